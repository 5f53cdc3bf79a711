"""What the drafted-step calls refuse, through the C ABI and the binding, before anything
reaches a GPU (the pointers are never followed)."""
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
    d = dict(num_blocks=10, block_size=16, num_kv_heads=2, head_size=64, dtype=pkv.PKV_BF16)
    d.update(kw)
    return pkv.CacheDesc(*d.values())


def rope_desc(**kw):
    d = dict(num_tokens=3, num_q_heads=4, num_kv_heads=2, head_size=64, dtype=pkv.PKV_BF16,
             rot_dim=64, max_position=100, interleaved=0, q_stride=256, k_stride=128, v_stride=128,
             q_out_stride=256, k_out_stride=128, eps=1e-6)
    d.update(kw)
    return pkv.RopeDesc(*d.values())


def meta(**kw):
    m = dict(num_seqs=1, num_tokens=3, num_q_heads=4, block_table_stride=2, max_query_len=3,
             max_context_len=20, num_decode_seqs=-1, sliding_window=0, kv_split_tokens=0)
    m.update(kw)
    return pkv.AttnMeta(*m.values())


def write(lib, r=None, c=None, **at):
    args = dict.fromkeys("q_out q k v pos cs qw kw slots kc vc".split(), P)
    args.update(at)
    return lib.pkv_rope_write(*args.values(), ctypes.byref(r or rope_desc()),
                              ctypes.byref(c or desc()), None)


def write_fp8(lib, r=None, c=None, **at):
    args = dict.fromkeys("q_out q k v pos cs qw kw slots kc vc ks vs".split(), P)
    args.update(at)
    return lib.pkv_rope_write_fp8(*args.values(), ctypes.byref(r or rope_desc()),
                                  ctypes.byref(c or desc(dtype=pkv.PKV_FP8_E4M3)), None)


def rows(lib, r=None, **at):
    args = dict.fromkeys("q_out k_out q k pos cs qw kw".split(), P)
    args.update(at)
    return lib.pkv_rope(*args.values(), ctypes.byref(r or rope_desc()), None)


def tree(lib, c=None, m=None, **at):
    args = dict.fromkeys("out q kc vc bt cl qsl mask".split(), P)
    args.update(at)
    return lib.pkv_attention_tree(*args.values(), 0.1, ctypes.byref(c or desc()),
                                  ctypes.byref(m or meta()), None, 0, None)


def tree_fp8(lib, c=None, m=None, **at):
    args = dict.fromkeys("out q kc vc bt cl qsl mask".split(), P)
    scales = dict(kd=P, vd=P)
    for n, x in at.items():
        (scales if n in scales else args)[n] = x
    return lib.pkv_attention_tree_fp8(*args.values(), 0.1, *scales.values(),
                                      ctypes.byref(c or desc(dtype=pkv.PKV_FP8_E4M3)),
                                      ctypes.byref(m or meta()), None, 0, None)


def accept(lib, nbuf=2, nb=10, stride=2, seqs=1, most=4, row=(256, 256), ptr=(P, P), **at):
    args = dict(bt=P, cl=P, qsl=P + 4096, acc=P, num=P, new=P + 8192)
    args.update(at)
    bufs = (ctypes.c_void_p * 2)(*ptr)
    rb = (ctypes.c_int64 * 2)(*row)
    return lib.pkv_accept_drafts(bufs, rb, nbuf, nb, args["bt"], stride, args["cl"], args["qsl"],
                                 seqs, args["acc"], args["num"], most, args["new"], None)


@pytest.mark.parametrize("call", [write, write_fp8, rows])
def test_rope_descriptions(lib, call):
    for bad in (dict(head_size=96), dict(num_tokens=-1), dict(num_q_heads=0), dict(num_kv_heads=0),
                dict(rot_dim=65), dict(rot_dim=63), dict(rot_dim=-2), dict(max_position=-1),
                dict(num_q_heads=65535), dict(q_stride=255), dict(k_stride=127),
                dict(q_out_stride=0), dict(q_stride=-256)):
        assert call(lib, r=rope_desc(**bad)) == E_SHAPE, bad
    assert call(lib, r=rope_desc(dtype=pkv.PKV_INT8)) == E_DTYPE
    for bad in (dict(q_stride=257), dict(k_stride=132)):
        assert call(lib, r=rope_desc(**bad)) == E_ALIGN, bad
    assert call(lib, r=rope_desc(num_tokens=0), q=None, pos=None) == 0


def test_rope_caches(lib):
    for c in (desc(num_kv_heads=3), desc(head_size=128), desc(block_size=8)):
        assert write(lib, c=c) == E_SHAPE
    assert write(lib, c=desc(dtype=pkv.PKV_F32)) == E_DTYPE
    assert write(lib, c=desc(dtype=pkv.PKV_FP8_E4M3)) == E_DTYPE
    assert write(lib, c=desc(dtype=pkv.PKV_INT8)) == E_DTYPE
    assert write_fp8(lib, c=desc()) == E_DTYPE
    assert write_fp8(lib, r=rope_desc(dtype=pkv.PKV_F32)) == E_DTYPE
    assert write(lib, r=rope_desc(v_stride=64)) == E_SHAPE
    assert rows(lib, r=rope_desc(k_out_stride=64)) == E_SHAPE


@pytest.mark.parametrize("call,names", [
    (write, "q_out q k v pos cs slots kc vc"), (write_fp8, "q_out q k v pos cs slots kc vc ks vs"),
    (rows, "q_out k_out q k pos cs"), (tree, "out q kc vc bt cl qsl mask"),
    (tree_fp8, "out q kc vc bt cl qsl mask kd vd"), (accept, "bt cl qsl acc num")])
def test_missing_pointers(lib, call, names):
    for n in names.split():
        assert call(lib, **{n: None}) == E_NULL, n


@pytest.mark.parametrize("call,names", [
    (write, "q_out q k v pos cs qw kw slots kc vc"), (rows, "q_out k_out q k pos cs qw kw"),
    (tree, "out q kc vc bt cl qsl mask"), (accept, "bt cl qsl acc num new")])
def test_unaligned_pointers(lib, call, names):
    for n in names.split():
        assert call(lib, **{n: P + 2}) == E_ALIGN, n


@pytest.mark.parametrize("call", [tree, tree_fp8])
def test_tree_descriptions(lib, call):
    fp8 = dict(dtype=pkv.PKV_FP8_E4M3) if call is tree_fp8 else {}
    for bad in (dict(block_size=32), dict(head_size=96), dict(num_kv_heads=0)):
        assert call(lib, c=desc(**{**fp8, **bad})) == E_SHAPE
    assert call(lib, c=desc(dtype=pkv.PKV_INT8)) == E_DTYPE
    assert call(lib, c=desc(dtype=pkv.PKV_BF16 if fp8 else pkv.PKV_FP8_E4M3)) == E_DTYPE
    assert call(lib, m=meta(num_q_heads=5)) == E_GQA
    for bad in (dict(sliding_window=8), dict(num_seqs=-1), dict(block_table_stride=0),
                dict(kv_split_tokens=63), dict(max_context_len=-1)):
        assert call(lib, m=meta(**bad)) == E_META, bad
    for bad in (dict(num_seqs=65536), dict(max_query_len=32 * 65536)):
        assert call(lib, m=meta(**bad)) == E_SHAPE, bad
    for empty in (dict(num_seqs=0), dict(num_tokens=0), dict(max_query_len=0)):
        assert call(lib, m=meta(**empty), q=None) == 0


def test_accept_descriptions(lib):
    for bad in (dict(nbuf=-1), dict(nb=-1), dict(seqs=-1), dict(most=-1), dict(nb=1 << 28),
                dict(row=(256, 0)), dict(row=(1 << 27, 256))):
        assert accept(lib, **bad) == E_SHAPE, bad
    assert accept(lib, stride=0) == E_META
    assert accept(lib, row=(256, 254)) == E_ALIGN
    assert accept(lib, ptr=(P, P + 2)) == E_ALIGN
    assert accept(lib, ptr=(P, None)) == E_NULL
    assert accept(lib, seqs=0, bt=None) == 0
    # the new lengths over the old ones, whole or in part
    assert accept(lib, new=P) == E_META
    assert accept(lib, seqs=4, new=P + 12) == E_META
    assert accept(lib, seqs=4, new=P - 12) == E_META


def test_new_lengths_over_other_arrays(lib):
    """Every CTA of a sequence reads these while the first writes the new length."""
    new = P + (1 << 16)
    for name, size in (("num", 16), ("qsl", 20), ("acc", 64), ("bt", 32)):
        for at in (new, new + 12, new - size + 4):
            assert accept(lib, seqs=4, new=new, **{name: at}) == E_META, (name, at)


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    T, hq, hkv, d = 3, 4, 2, 64
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    q, k = b(T, hq, d), b(T, hkv, d)
    pos, cs = torch.zeros(T, dtype=torch.int64), torch.zeros(10, d)
    cache = b(4, 16, hkv, d)
    with pytest.raises(pkv.PkvError):
        pkv.rope(q, k, q, k, pos, cs)
    with pytest.raises(pkv.PkvError):
        pkv.rope_write(q, q, k, k, pos, cs, pos, cache, cache)
    with pytest.raises(pkv.PkvError):
        pkv.rope_write_fp8(q, q, k, k, pos, cs, pos, cache, cache, torch.ones(hkv), torch.ones(hkv))
    with pytest.raises(pkv.PkvError, match="num_tokens"):
        pkv.rope(q[0], k, q[0], k, pos, cs)
    with pytest.raises(pkv.PkvError, match="unsupported"):
        pkv.rope(q.half(), k.half(), q.half(), k.half(), pos, cs)
    mask = torch.zeros(T, 1, dtype=torch.int64)
    tree = lambda c, fn=pkv.attention_tree, *more: fn(
        q, q, c, c, i32(1, 2), i32(1), i32(2), mask, 0.1, *more, max_query_len=T,
        max_context_len=20)
    with pytest.raises(pkv.PkvError, match="CUDA"):
        tree(cache)
    with pytest.raises(pkv.PkvError, match="int8"):
        tree(cache.to(torch.int8))
    with pytest.raises(pkv.PkvError, match="e4m3"):
        tree(cache, pkv.attention_tree_fp8, torch.ones(1, hkv), torch.ones(1, hkv))
    with pytest.raises(pkv.PkvError):
        pkv.accept_drafts([cache], i32(1, 2), i32(1), i32(2), i32(1, 4), i32(1))


def test_groups_past_a_tile(lib):
    """More q heads on a kv head than a tile has rows (fp32 takes them)."""
    assert tree(lib, m=meta(num_q_heads=2 * 129)) == E_SHAPE
    assert tree_fp8(lib, m=meta(num_q_heads=2 * 129)) == E_SHAPE


def test_rope_struct_layout_matches_header(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pkv.h"\n'
                   'int main(void){printf("%zu %zu %zu\\n", sizeof(pkv_rope_desc), '
                   'offsetof(pkv_rope_desc, q_stride), offsetof(pkv_rope_desc, eps));return 0;}\n')
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o",
                    str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(pkv.RopeDesc), pkv.RopeDesc.q_stride.offset,
                                     pkv.RopeDesc.eps.offset]
