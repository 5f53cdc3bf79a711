"""The rotation calls over so many tokens that a CTA walks several (the next one's rows, position and slot are
on their way while one is computed), against 64-bit references."""
import pytest
import torch

from drafts import EPS, rope_reference
from paged_kv_cache_43_gb300 import build, pkv

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
POSITIONS = 500
# rotated elements and pairing: half rotations in whole chunks, and anyhow; neighbours
ROTS = [(64, 64, False), (64, 6, False), (64, 6, True), (128, 128, False), (128, 90, False), (128, 32, True)]
# tokens such that the GPU's CTAs walk two and three each
SIZES = [(9001, 3, 1), (2011, 8, 2), (1009, 32, 8)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    pkv.load()
    pkv.get_error(clear=True)
    yield
    assert pkv.get_error(clear=True) == 0


class Rows:
    def __init__(self, T, hq, hkv, d, dtype, rot, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: (torch.randn(s, generator=g, device="cuda") * 1.5).to(dtype)
        self.x = rand(T, (hq + 2 * hkv) * d + 16)     # (rows of q, k, v and something else)
        self.q, self.k, self.v = (t.view(T, -1, d) for t in self.x[:, :-16].split(
            [hq * d, hkv * d, hkv * d], 1))
        self.qw, self.kw = rand(d), rand(d)
        f = 10000.0 ** -(torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))
        a = torch.arange(POSITIONS, dtype=torch.float64)[:, None] * f
        self.cs = torch.cat([a.cos(), a.sin()], 1).float().cuda()
        self.pos = torch.randint(0, POSITIONS, (T,), generator=g, device="cuda")
        self.nb = -(-T // 16) + 2
        self.slots = torch.randperm(self.nb * 16, generator=g, device="cuda")[:T]
        self.args = dict(q_weight=self.qw, k_weight=self.kw, eps=1e-5)

    def want(self, interleaved):
        return [rope_reference(x, w, 1e-5, self.cs, self.pos.clamp(0, POSITIONS - 1), interleaved)
                for x, w in ((self.q, self.qw), (self.k, self.kw))]

    def leave_out(self):
        """Padding, slots past the cache and positions outside the table, all through the batch."""
        T = len(self.slots)
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        for first, step, what in ((3, 7, "pad"), (5, 31, "slot"), (11, 29, "pos"), (12, 37, "neg")):
            at = torch.arange(first, T, step, device="cuda")
            keep[at] = False
            if what == "pad":
                self.slots[at] = -1
            elif what == "slot":
                self.slots[at] = self.nb * 16 + 3
            else:
                self.pos[at] = POSITIONS if what == "pos" else -4
        return keep


def close(got, want, tol, dtype):
    off = (got.double() - want).abs() - tol - EPS[dtype] * want.abs()
    assert float(off.max()) <= 0, f"{float(off.max()):.3e} past the bound"


@pytest.mark.parametrize("T,hq,hkv", SIZES)
@pytest.mark.parametrize("d,rot,interleaved", ROTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gaps", [False, True])
def test_write(T, hq, hkv, d, rot, interleaved, dtype, gaps):
    r = Rows(T, hq, hkv, d, dtype, rot, seed=T + rot)
    at = r.slots.clone()
    keep = r.leave_out() if gaps else torch.ones(T, dtype=torch.bool, device="cuda")
    kc = torch.full((r.nb, 16, hkv, d), 3.0, dtype=dtype, device="cuda")
    vc = kc.clone()
    wide = torch.full((T, hq * d + 32), 7.0, dtype=dtype, device="cuda")
    out = wide[:, :-32].view(T, hq, d)
    pkv.rope_write(out, r.q, r.k, r.v, r.pos, r.cs, r.slots, kc, vc, interleaved=interleaved, **r.args)
    assert pkv.get_error() == (pkv.ERR_SLOT | pkv.ERR_POSITION if gaps else 0)
    (q, qt), (k, kt) = r.want(interleaved)
    kr, vr = kc.flatten(0, 1), vc.flatten(0, 1)
    close(out[keep], q[keep], qt[keep], dtype)
    close(kr[at[keep]], k[keep], kt[keep], dtype)
    assert torch.equal(vr[at[keep]], r.v[keep])
    rest = torch.ones(r.nb * 16, dtype=torch.bool, device="cuda")
    rest[at[keep]] = False
    assert bool((kr[rest] == 3.0).all()) and bool((vr[rest] == 3.0).all())
    assert bool((out[~keep] == 7.0).all()) and bool((wide[:, -32:] == 7.0).all())


@pytest.mark.parametrize("T,hq,hkv", SIZES)
@pytest.mark.parametrize("d,rot,interleaved", ROTS)
def test_write_fp8(T, hq, hkv, d, rot, interleaved):
    r = Rows(T, hq, hkv, d, BF16, rot, seed=T + rot)
    at = r.slots.clone()
    keep = r.leave_out()
    kc = torch.full((r.nb, 16, hkv, d), 3.0, device="cuda").to(E4M3)
    vc = kc.clone()
    ks, vs = (torch.rand(hkv, device="cuda") * 0.02 + 0.003 for _ in range(2))
    out = torch.full((T, hq, d), 7.0, dtype=BF16, device="cuda")
    pkv.rope_write_fp8(out, r.q, r.k, r.v, r.pos, r.cs, r.slots, kc, vc, ks, vs,
                       interleaved=interleaved, **r.args)
    assert pkv.get_error() == pkv.ERR_SLOT | pkv.ERR_POSITION
    (q, qt), (k, kt) = r.want(interleaved)
    close(out[keep], q[keep], qt[keep], BF16)
    assert bool((out[~keep] == 7.0).all())
    codes = lambda c: c.view(torch.uint8).flatten(0, 1)
    got = codes(kc)[at[keep]].view(E4M3).double()
    s = ks.double()[:, None]
    want = (k[keep] / s).clamp(-448, 448)
    # half a step of a value (2^-4) or of the smallest ones (2^-10), the arithmetic's error
    assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 + kt[keep] / s
                 + want.abs() * 2.0 ** -22).all())
    k2 = torch.full_like(kc.view(torch.uint8), 9).view(E4M3)      # v: the codes that pkv_write_fp8 makes
    v2 = k2.clone()
    pkv.write_fp8(r.v.contiguous(), r.v.contiguous(), torch.where(keep, at, -1), k2, v2, ks, vs)
    assert torch.equal(codes(vc)[at[keep]], codes(v2)[at[keep]])
    rest = torch.ones(r.nb * 16, dtype=torch.bool, device="cuda")
    rest[at[keep]] = False
    for c in (kc, vc):
        assert bool((codes(c)[rest].view(E4M3).float() == 3.0).all())


@pytest.mark.parametrize("T,hq,hkv", SIZES)
@pytest.mark.parametrize("d,rot,interleaved", ROTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_alone_and_in_place(T, hq, hkv, d, rot, interleaved, dtype):
    r = Rows(T, hq, hkv, d, dtype, rot, seed=T + rot)
    at = torch.arange(11, T, 29, device="cuda")
    r.pos[at] = POSITIONS + 1
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[at] = False
    (q, qt), (k, kt) = r.want(interleaved)
    qo = torch.full((T, hq, d), 7.0, dtype=dtype, device="cuda")
    ko = torch.full((T, hkv, d), 7.0, dtype=dtype, device="cuda")
    pkv.rope(qo, ko, r.q, r.k, r.pos, r.cs, interleaved=interleaved, **r.args)
    assert pkv.get_error() == pkv.ERR_POSITION
    close(qo[keep], q[keep], qt[keep], dtype)
    close(ko[keep], k[keep], kt[keep], dtype)
    assert bool((qo[~keep] == 7.0).all()) and bool((ko[~keep] == 7.0).all())
    x = r.x.clone()
    pkv.rope(r.q, r.k, r.q, r.k, r.pos, r.cs, interleaved=interleaved, **r.args)   # over the rows themselves
    assert pkv.get_error() == pkv.ERR_POSITION
    assert torch.equal(r.q[keep], qo[keep]) and torch.equal(r.k[keep], ko[keep])
    assert torch.equal(r.x[~keep], x[~keep])
    assert torch.equal(r.v, x[:, (hq + hkv) * d:-16].view(T, hkv, d)) and torch.equal(r.x[:, -16:], x[:, -16:])
