"""pkv_rope_write, pkv_rope_write_fp8 and pkv_rope against 64-bit references."""
import numpy as np
import pytest
import torch

from drafts import EPS, rope_reference
from paged_kv_cache_43_gb300 import build, pkv

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    pkv.load()
    pkv.get_error(clear=True)
    yield
    assert pkv.get_error(clear=True) == 0


def table(n, rot):
    f = 10000.0 ** -(torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


class Rows:
    def __init__(self, T, hq, hkv, d, dtype, rot, *, norm=True, packed=True, seed=0, positions=200):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: (torch.randn(s, generator=g, device="cuda") * 1.5).to(dtype)
        if packed:
            x = rand(T, (hq + 2 * hkv) * d)
            self.q, self.k, self.v = (t.view(T, -1, d) for t in
                                      x.split([hq * d, hkv * d, hkv * d], 1))
        else:
            self.q, self.k, self.v = rand(T, hq, d), rand(T, hkv, d), rand(T, hkv, d)
        self.qw, self.kw = (rand(d), rand(d)) if norm else (None, None)
        self.cs = table(positions, rot)
        self.pos = torch.randint(0, positions, (T,), generator=g, device="cuda")
        nb = -(-T // 16) + 2
        self.slots = torch.randperm(nb * 16, generator=g, device="cuda")[:T]
        self.cache_shape = (nb, 16, hkv, d)
        self.kw_args = dict(q_weight=self.qw, k_weight=self.kw, eps=1e-5)

    def want(self, interleaved):
        return [rope_reference(x, w, 1e-5, self.cs, self.pos, interleaved)
                for x, w in ((self.q, self.qw), (self.k, self.kw))]


def close(got, want, tol, dtype):
    off = (got.double() - want).abs() - tol - EPS[dtype] * want.abs()
    assert float(off.max()) <= 0, f"{float(off.max()):.3e} past the bound"


def caches(r, dtype):
    x = torch.full(r.cache_shape, 3.0, device="cuda").to(dtype)
    return x, x.clone()


@pytest.mark.parametrize("T,hq,hkv", [(1, 32, 8), (7, 4, 4), (333, 3, 1), (65, 40, 8), (2, 1, 1)])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 6), (128, 128), (128, 32), (128, 90)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_write(T, hq, hkv, d, rot, interleaved):
    for dtype in (torch.bfloat16, torch.float32):
        r = Rows(T, hq, hkv, d, dtype, rot, seed=T + d, packed=rot % 4 == 0)
        kc, vc = caches(r, dtype)
        out = torch.zeros((T, hq, d), dtype=dtype, device="cuda")
        pkv.rope_write(out, r.q, r.k, r.v, r.pos, r.cs, r.slots, kc, vc, interleaved=interleaved,
                       **r.kw_args)
        (q, qt), (k, kt) = r.want(interleaved)
        close(out, q, qt, dtype)
        close(kc.flatten(0, 1)[r.slots], k, kt, dtype)
        assert torch.equal(vc.flatten(0, 1)[r.slots], r.v)
        rest = torch.ones(kc.shape[0] * 16, dtype=torch.bool, device="cuda")
        rest[r.slots] = False
        for c in (kc, vc):
            assert bool((c.flatten(0, 1)[rest] == 3.0).all())


@pytest.mark.parametrize("T,hq,hkv,d,rot", [(1, 8, 2, 128, 128), (50, 15, 5, 64, 32),
                                            (129, 2, 2, 128, 10), (40, 1, 3, 64, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_write_fp8(T, hq, hkv, d, rot, interleaved):
    r = Rows(T, hq, hkv, d, torch.bfloat16, rot, seed=T)
    kc, vc = caches(r, E4M3)
    ks, vs = (torch.rand(hkv, device="cuda") * 0.02 + 0.003 for _ in range(2))
    out = torch.zeros((T, hq, d), dtype=torch.bfloat16, device="cuda")
    pkv.rope_write_fp8(out, r.q, r.k, r.v, r.pos, r.cs, r.slots, kc, vc, ks, vs,
                       interleaved=interleaved, **r.kw_args)
    (q, qt), (k, kt) = r.want(interleaved)
    close(out, q, qt, torch.bfloat16)
    got = kc.view(torch.uint8).flatten(0, 1)[r.slots].view(E4M3).double()
    s = ks.double()[:, None]
    want = (k / s).clamp(-448, 448)
    # half a step of a value (2^-4) or of the smallest ones (2^-10), the arithmetic's error
    assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 + kt / s
                 + want.abs() * 2.0 ** -22).all())
    # v: the codes that pkv_write_fp8 makes
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    pkv.write_fp8(r.v.contiguous(), r.v.contiguous(), r.slots, k2, v2, ks, vs)
    at = lambda c: c.view(torch.uint8).flatten(0, 1)[r.slots]
    assert torch.equal(at(vc), at(v2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_alone_and_in_place(dtype):
    r = Rows(37, 6, 2, 128, dtype, 64)
    (q, qt), (k, kt) = r.want(False)
    qo, ko = torch.empty_like(q, dtype=dtype), torch.empty_like(k, dtype=dtype)
    pkv.rope(qo, ko, r.q, r.k, r.pos, r.cs, **r.kw_args)
    close(qo, q, qt, dtype)
    close(ko, k, kt, dtype)
    v = r.v.clone()
    pkv.rope(r.q, r.k, r.q, r.k, r.pos, r.cs, **r.kw_args)    # over the packed rows themselves
    assert torch.equal(r.q, qo) and torch.equal(r.k, ko) and torch.equal(r.v, v)


def test_without_norms_or_with_one():
    r = Rows(20, 4, 2, 64, torch.bfloat16, 64)
    for qw, kw in ((None, None), (r.qw, None), (None, r.kw)):
        r.qw, r.kw, keep = qw, kw, (r.qw, r.kw)
        (q, qt), (k, kt) = r.want(False)
        qo, ko = torch.empty_like(q, dtype=r.q.dtype), torch.empty_like(k, dtype=r.q.dtype)
        pkv.rope(qo, ko, r.q, r.k, r.pos, r.cs, q_weight=qw, k_weight=kw, eps=1e-5)
        close(qo, q, qt, r.q.dtype)
        close(ko, k, kt, r.q.dtype)
        r.qw, r.kw = keep


def test_padding_and_bad_tokens_are_left_alone():
    """-1 slots, slots past the cache, positions outside the table: nothing of them is written,
    and the others are."""
    r = Rows(40, 4, 2, 64, torch.bfloat16, 64)
    kc, vc = caches(r, torch.bfloat16)
    out = torch.full((40, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    before = r.slots.clone()
    r.slots[3] = -1
    r.slots[4] = kc.shape[0] * 16
    r.pos[5], r.pos[6] = -1, 200
    r.pos[7], r.slots[7] = 1 << 40, -5       # (padding is not looked at)
    good = torch.ones(40, dtype=torch.bool, device="cuda")
    good[3:8] = False
    pkv.rope_write(out, r.q, r.k, r.v, r.pos, r.cs, r.slots, kc, vc, **r.kw_args)
    assert pkv.get_error() == pkv.ERR_SLOT | pkv.ERR_POSITION
    r.pos[~good] = 0
    (q, qt), (k, kt) = r.want(False)
    close(out[good], q[good], qt[good], torch.bfloat16)
    assert bool((out[~good] == 7.0).all())
    rows = kc.flatten(0, 1)
    close(rows[before[good]], k[good], kt[good], torch.bfloat16)
    assert bool((rows[before[~good]] == 3.0).all())


def test_not_finite_values_stay_in_their_head():
    r = Rows(3, 4, 2, 64, torch.bfloat16, 64, packed=False)
    r.q[1, 2, 5] = float("inf")
    r.k[0, 1, 60] = float("nan")
    qo, ko = torch.empty_like(r.q), torch.empty_like(r.k)
    pkv.rope(qo, ko, r.q, r.k, r.pos, r.cs, **r.kw_args)
    bad_q, bad_k = torch.isfinite(qo).all(2), torch.isfinite(ko).all(2)
    assert not bad_q[1, 2] and int(bad_q.sum()) == 11
    assert not bad_k[0, 1] and int(bad_k.sum()) == 5


def test_graph_replay_and_stream():
    r = Rows(64, 8, 2, 128, torch.bfloat16, 128)
    kc, vc = caches(r, torch.bfloat16)
    out = torch.zeros((64, 8, 128), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (out, r.q, r.k, r.v, r.pos, r.cs, r.slots, kc, vc)
    pkv.rope_write(*args, stream=s, **r.kw_args)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.rope_write(*args, **r.kw_args)
    r.q.normal_()
    r.pos.random_(0, 200)
    g.replay()
    (q, qt), (k, kt) = r.want(False)
    close(out, q, qt, torch.bfloat16)
    close(kc.flatten(0, 1)[r.slots], k, kt, torch.bfloat16)


def test_offsets_past_32_bits():
    """Slots of a cache of more than 2^31 elements, rows further apart than that."""
    hkv, d, T = 8, 128, 4
    nb = (1 << 31) // (16 * hkv * d) + 8
    r = Rows(T, 4, hkv, d, torch.bfloat16, 128)
    kc = torch.zeros((nb, 16, hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    r.slots = torch.tensor([0, nb * 16 - 1, nb * 16 - 77, 5], device="cuda")
    out = torch.zeros((T, 4, d), dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros(3 * (1 << 30) + 4 * d, dtype=torch.bfloat16, device="cuda")
    q = wide.as_strided((T, 4, d), (1 << 30, d, 1))
    q.copy_(r.q)
    pkv.rope_write(out, q, r.k, r.v, r.pos, r.cs, r.slots, kc, vc, **r.kw_args)
    (qq, qt), (k, kt) = r.want(False)
    close(out, qq, qt, torch.bfloat16)
    close(kc.view(-1, hkv, d)[r.slots], k, kt, torch.bfloat16)
    assert torch.equal(vc.view(-1, hkv, d)[r.slots], r.v)


def test_no_tokens():
    r = Rows(1, 4, 2, 64, torch.bfloat16, 64)
    kc, vc = caches(r, torch.bfloat16)
    e = lambda t: t[:0]
    pkv.rope_write(e(r.q), e(r.q), e(r.k), e(r.v), e(r.pos), r.cs, e(r.slots), kc, vc)
    assert bool((kc == 3.0).all())


def test_refusals_of_gpu_tensors():
    r = Rows(5, 4, 2, 64, torch.bfloat16, 64)
    kc, vc = caches(r, torch.bfloat16)
    out = torch.zeros((5, 4, 64), dtype=torch.bfloat16, device="cuda")
    call = lambda **kw: pkv.rope_write(*{**dict(q_out=out, q=r.q, k=r.k, v=r.v, pos=r.pos, cs=r.cs,
                                                slots=r.slots, kc=kc, vc=vc), **kw}.values())
    for bad in (dict(q=r.q.transpose(0, 1)), dict(q=r.q[:4]), dict(v=r.k[:, :1]),
                dict(pos=r.pos.int()), dict(slots=r.slots[:3]), dict(cs=r.cs.double()),
                dict(kc=kc.float()), dict(vc=vc[:1]), dict(cs=torch.zeros(9, 200, device="cuda")),
                dict(cs=torch.zeros(9, 63, device="cuda")), dict(q=r.q.cpu()),
                dict(q=r.q[:1].expand(5, 4, 64))):
        with pytest.raises(pkv.PkvError):
            call(**bad)
    with pytest.raises(pkv.PkvError):
        pkv.rope_write(out, r.q, r.k, r.v, r.pos, r.cs, r.slots, kc, vc, q_weight=r.qw.float())
