"""Host-side checks of rotary positions, the residual norm and the gated linear layer that need no GPU: bad arguments are rejected
before anything is enqueued, so fake device pointers are never touched; workspace sizes; frequencies."""
import math
import os

import pytest
import torch

FAKE = 1 << 40        # 16-byte aligned, never dereferenced: every case fails validation first
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    import dense_descriptor_matching_amd as ddm
    if not os.path.exists(ddm.LIB_PATH):
        pytest.fail("libddm.so not built: run __graft_entry__.build()")
    return ddm.lib()


def _rotary(L, **kw):
    a = dict(q=FAKE, qt=256, qh=64, Hq=4, k=FAKE, kt=128, kh=64, Hk=2, pos=FAKE, freq=FAKE, T=10, D=64, axes=2, pairs=16, dtype=1,
             interleaved=0, inverse=0, m=1.0, qo=FAKE, qot=256, qoh=64, ko=FAKE, kot=128, koh=64)
    a.update(kw)
    return L.ddm_rotary(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1), (dict(ko=None), -1), (dict(q=FAKE + 1), -1), (dict(ko=FAKE + 1), -1),
    (dict(pos=None), -1), (dict(pos=FAKE + 2), -1), (dict(freq=None), -1), (dict(freq=FAKE + 4), -1), (dict(T=-1), -1), (dict(D=0), -4),
    (dict(D=1025), -4), (dict(D=63), -1), (dict(axes=0), -1), (dict(pairs=0), -1), (dict(pairs=17), -1), (dict(axes=3), -1),
    (dict(axes=1 << 30, pairs=1 << 30), -1), (dict(dtype=3), -4), (dict(interleaved=2), -1), (dict(inverse=-1), -1),
    (dict(m=float("nan")), -1), (dict(m=1e39), -1), (dict(Hq=-1), -1), (dict(Hk=65537), -1), (dict(qt=-1), -1), (dict(koh=-64), -1),
    (dict(kt=1 << 41), -1), (dict(qot=0), -1), (dict(koh=0), -1)])
def test_rotary_rejects(L, change, status):
    assert _rotary(L, **change) == status


def test_rotary_with_nothing_to_do(L):
    assert _rotary(L, T=0, q=None, k=None) == 0
    assert _rotary(L, Hq=0, Hk=0, q=None, k=None, qo=None, ko=None) == 0


def test_frequencies():
    import dense_descriptor_matching_amd as ddm
    f = ddm.rotary_frequencies(32)
    i = torch.arange(32, dtype=torch.float64)
    assert f.dtype == torch.float64 and torch.allclose(f, 10000.0 ** (-i / 32), rtol=1e-14)
    assert torch.equal(ddm.rotary_frequencies(32, scaling="linear", factor=4.0), f / 4)
    b = ddm.rotary_frequencies(32, scaling="base", factor=4.0)
    assert b[0] == 1 and abs(b[-1] / (f[-1] / 4) - 1) < 1e-12 and (b <= f).all()
    r = ddm.rotary_frequencies(32, scaling="ramp", factor=4.0, length=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(r[turns >= 32], f[turns >= 32]) and torch.equal(r[turns <= 1], (f / 4)[turns <= 1])
    assert ((r < f) & (r > f / 4))[(turns > 1) & (turns < 32)].all() and (r.diff() < 0).all()
    assert ddm.rotary_frequencies(1, scaling="base", factor=4.0).tolist() == [1.0]
    for bad in (dict(pairs=0), dict(pairs=4, base=0.0), dict(pairs=4, factor=-1.0), dict(pairs=4, scaling="ramp"),
                dict(pairs=4, scaling="ramp", length=10, slow=5.0, fast=5.0), dict(pairs=4, scaling="other")):
        with pytest.raises(ValueError):
            ddm.rotary_frequencies(**bad)


def _norm(L, **kw):
    a = dict(x=FAKE, ldx=64, br=FAKE, ldb=64, gate=FAKE, ldg=64, scale=FAKE, bw=FAKE, bb=FAKE, w=FAKE, b=FAKE, N=10, C=64, dtype=2,
             wtype=0, bn=1, rms=0, eps=1e-6, s=FAKE, y=FAKE, stats=FAKE)
    a.update(kw)
    return L.ddm_residual_norm_forward(*a.values(), None)


def _norm_back(L, **kw):
    a = dict(dy=FAKE, ds=FAKE, x=FAKE, ldx=64, br=FAKE, ldb=64, gate=FAKE, ldg=64, scale=FAKE, bw=FAKE, bb=FAKE, w=FAKE, stats=FAKE, N=10,
             C=64, dtype=2, wtype=0, bn=1, rms=0, dx=FAKE, dbr=FAKE, dg=FAKE, dsc=FAKE, dbw=FAKE, dbb=FAKE, dw=FAKE, db=FAKE, ws=FAKE,
             wsb=BIG)
    a.update(kw)
    return L.ddm_residual_norm_backward(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), -1), (dict(br=None), -1), (dict(x=FAKE + 1), -1), (dict(br=FAKE + 1), -1), (dict(gate=FAKE + 1), -1), (dict(ldx=63), -1),
    (dict(ldb=63), -1), (dict(ldg=63), -1), (dict(N=-1), -1), (dict(N=1 << 32), -1), (dict(C=0), -4), (dict(C=8193), -4),
    (dict(dtype=7), -4), (dict(wtype=1), -4), (dict(stats=None), -1), (dict(stats=FAKE + 2), -1), (dict(w=FAKE + 2), -1),
    (dict(scale=FAKE + 2), -1), (dict(bw=FAKE + 2), -1), (dict(bb=FAKE + 2), -1), (dict(bn=2), -1), (dict(rms=2), -1), (dict(bn=0), -1)])
def test_residual_norm_rejects(L, change, status):
    assert _norm(L, **change) == status
    assert _norm_back(L, **change) == status


def test_residual_norm_rejects_one_way(L):
    assert _norm(L, s=None) == -1 and _norm(L, y=None) == -1 and _norm(L, b=FAKE + 2) == -1
    for eps in (-1.0, float("nan"), float("inf"), 1e39):
        assert _norm(L, eps=eps) == -1
    assert _norm(L, N=0, x=None, y=None) == 0                       # nothing launched
    assert _norm_back(L, ws=None) == -3 and _norm_back(L, wsb=16) == -3 and _norm_back(L, ws=FAKE + 4) == -3
    assert _norm_back(L, gate=None) == -1                           # the gradient of a gate that is not there
    for n in ("dy", "ds", "dx", "dbr", "dg", "dw", "dsc"):
        assert _norm_back(L, **{n: FAKE + 1}) == -1
    none = dict(dsc=None, dbw=None, dbb=None, dw=None, db=None)
    assert _norm_back(L, N=0, ws=None, **none) == 0
    assert _norm_back(L, dx=None, dbr=None, dg=None, ws=None, **none) == 0
    f = L.ddm_residual_norm_backward_workspace_bytes
    assert f(100, 9000, 0, 0) == 0 and f(-1, 64, 0, 0) == 0 and f(10, 64, 5, 0) == 0
    assert f(100000, 1024, 2, 1) > f(100000, 1024, 2, 0) >= 3 * 1024 * 4 and f(0, 64, 0, 0) >= 3 * 64 * 4


def _gated(L, **kw):
    a = dict(x=FAKE, ldx=64, w=FAKE, b=FAKE, N=100, C=64, F=48, dtype=1, act=0, h=FAKE, kept=FAKE, ws=FAKE, wsb=BIG)
    a.update(kw)
    return L.ddm_gated_linear_forward(*a.values(), None)


def _gated_back(L, **kw):
    a = dict(dh=FAKE, x=FAKE, ldx=64, w=FAKE, kept=FAKE, N=100, C=64, F=48, dtype=1, act=0, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, wsb=BIG)
    a.update(kw)
    return L.ddm_gated_linear_backward(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), -1), (dict(x=FAKE + 1), -1), (dict(w=None), -1), (dict(w=FAKE + 8), -1), (dict(ldx=63), -1), (dict(ldx=1 << 22), -1),
    (dict(N=-1), -1), (dict(N=(1 << 24) + 1), -1), (dict(C=0), -4), (dict(F=0), -4), (dict(C=262145, ldx=262145), -4), (dict(F=262145), -4),
    (dict(dtype=3), -4), (dict(act=3), -1), (dict(act=-1), -1), (dict(kept=FAKE + 1), -1), (dict(ws=None), -3), (dict(ws=FAKE + 4), -3),
    (dict(wsb=15), -3), (dict(C=8192, ldx=8192, F=65536), -1), (dict(N=1 << 24, F=1 << 14), -1)])
def test_gated_linear_rejects(L, change, status):
    assert _gated(L, **change) == status
    assert _gated_back(L, **change) == status


def test_gated_linear_rejects_one_way(L):
    assert _gated(L, h=None) == -1 and _gated(L, b=FAKE + 1) == -1
    assert _gated_back(L, dh=None) == -1 and _gated_back(L, kept=None) == -1
    for n in ("dx", "dw", "db"):
        assert _gated_back(L, **{n: FAKE + 1}) == -1
    assert _gated(L, N=0, x=None, h=None, ws=None) == 0             # nothing launched
    assert _gated_back(L, dx=None, dw=None, db=None) == 0
    f, b = L.ddm_gated_linear_forward_workspace_bytes, L.ddm_gated_linear_backward_workspace_bytes
    for bad in ((-1, 64, 48, 1), (10, 0, 48, 1), (10, 64, 0, 1), (10, 64, 48, 4), (10, 1 << 19, 48, 1)):
        assert f(*bad) == 0 and b(*bad) == 0
    assert f(0, 64, 48, 1) > 0 and b(0, 64, 48, 1) > 0
    assert b(1000, 64, 48, 1) >= 1000 * 2 * 48 * 2                  # the projections' gradients
    assert f(1000, 61, 48, 1) >= (1000 + 96) * 64 * 2               # both operands repacked
    for N in (10, 1000, 10 ** 5, 10 ** 7):                          # of sums of tiles cut along k at most 128 MB
        for C, F in ((64, 64), (1024, 2736), (8192, 1000)):
            own = (N * C + 2 * N * F + 2 * F * C) * 2 + (N // 16 + 1) * 2 * F * 4
            assert b(N, C, F, 1) <= own + (1 << 27) + 4096 and f(N, C, F, 1) <= own + (1 << 27) + 4096
