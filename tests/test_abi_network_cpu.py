"""Host-side checks of the network operators' C ABI that need no GPU: bad arguments are rejected before anything is enqueued,
so fake device pointers are never touched, and workspace sizes follow the sizes."""
import os

import pytest

FAKE = 1 << 40        # 16-byte aligned, never dereferenced: every case fails validation first
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    import dense_descriptor_matching_amd as ddm
    if not os.path.exists(ddm.LIB_PATH):
        pytest.fail("libddm.so not built: run __graft_entry__.build()")
    return ddm.lib()


def _attn(L, backward=False, **kw):
    a = dict(g=FAKE, gt=256, gh=64, q=FAKE, qt=256, qh=64, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, out=FAKE, lse=FAKE,
             cq=FAKE, ck=FAKE, B=2, Tq=100, Tk=90, Hq=4, Hkv=2, D=64, dtype=1, causal=0, scale=0.125, dq=FAKE, dk=FAKE, dv=FAKE,
             ws=FAKE, wsb=BIG)
    a.update(kw)
    view = lambda *n: [a[x] for x in n]  # noqa: E731
    sizes = view("cq", "ck", "B", "Tq", "Tk", "Hq", "Hkv", "D", "dtype", "causal", "scale")
    if backward:
        return L.ddm_attention_backward(*view("g", "gt", "gh", "q", "qt", "qh", "k", "kt", "kh", "v", "vt", "vh", "out", "lse"),
                                        *sizes, *view("dq", "dk", "dv", "ws", "wsb"), None)
    return L.ddm_attention_forward(*view("q", "qt", "qh", "k", "kt", "kh", "v", "vt", "vh"), *sizes,
                                   *view("out", "lse", "ws", "wsb"), None)


BAD_ATTENTION = [(dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(q=FAKE + 8), -1), (dict(kt=132), -1),
                 (dict(vh=60), -1), (dict(qt=-256), -1), (dict(kt=1 << 23), -1), (dict(B=0), -1), (dict(Tq=-1), -1),
                 (dict(Hq=3), -1), (dict(Hkv=0), -1), (dict(D=0), -4), (dict(D=136), -4), (dict(D=60), -4), (dict(dtype=3), -4),
                 (dict(causal=2), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1),
                 (dict(scale=float("inf")), -1), (dict(cq=None), -1), (dict(ck=None), -1), (dict(Tq=1 << 30), -1),
                 (dict(lse=None), -1), (dict(out=None), -1)]


@pytest.mark.parametrize("change,status", BAD_ATTENTION)
def test_attention_rejects(L, change, status):
    assert _attn(L, **change) == status
    assert _attn(L, backward=True, **change) == status


def test_attention_workspace_and_gradient_pointers(L):
    assert _attn(L, backward=True, wsb=16) == -3
    assert _attn(L, backward=True, ws=None) == -3
    assert _attn(L, backward=True, ws=FAKE + 4) == -3
    assert _attn(L, backward=True, qh=1 << 28) == -1        # a group's heads beyond 31-bit offsets
    for n in ("g", "dq", "dk", "dv"):
        assert _attn(L, backward=True, **{n: None}) == -1
    assert _attn(L, Tq=2, Tk=5000, ws=None) == -3           # few rows over long keys: the parts lie in the workspace
    assert _attn(L, Tq=2, Tk=5000, wsb=64) == -3
    assert _attn(L, Tq=0, q=None, out=None, lse=None) == 0  # nothing to do, nothing launched


def test_attention_workspace_sizes(L):
    f, b = L.ddm_attention_forward_workspace_bytes, L.ddm_attention_backward_workspace_bytes
    assert 0 < f(2, 1536, 1536, 16, 16, 64, 1) <= 256       # whole rows need none
    assert f(2, 2, 80000, 16, 16, 64, 1) > 1 << 20
    assert f(2, 2, 80000, 16, 16, 64, 1) < 1 << 28
    assert b(2, 1536, 1536, 16, 16, 64, 1) > b(2, 1536, 1536, 16, 16, 64, 2) >= 1536 * 16 * 8
    for bad in ((0, 8, 8, 4, 2, 64, 1), (1, 8, 8, 3, 2, 64, 1), (1, 8, 8, 4, 2, 12, 1), (1, 8, 8, 4, 2, 64, 5)):
        assert f(*bad) == 0 and b(*bad) == 0


def _norm(L, **kw):
    a = dict(x=FAKE, ldx=64, w=FAKE, b=FAKE, N=10, C=64, dtype=2, wtype=0, eps=1e-6, y=FAKE, mean=FAKE, rstd=FAKE)
    a.update(kw)
    return L.ddm_layer_norm_forward(*a.values(), None)


def _norm_back(L, **kw):
    a = dict(dy=FAKE, x=FAKE, ldx=64, w=FAKE, mean=FAKE, rstd=FAKE, N=10, C=64, dtype=2, wtype=0, dx=FAKE, dw=FAKE, db=FAKE,
             ws=FAKE, wsb=BIG)
    a.update(kw)
    return L.ddm_layer_norm_backward(*a.values(), None)


@pytest.mark.parametrize("change,status", [(dict(x=None), -1), (dict(x=FAKE + 1), -1), (dict(ldx=63), -1), (dict(N=-1), -1),
                                           (dict(C=0), -4), (dict(C=8193), -4), (dict(dtype=7), -4), (dict(wtype=1), -4),
                                           (dict(mean=None), -1), (dict(rstd=FAKE + 2), -1), (dict(w=FAKE + 2), -1),
                                           (dict(N=1 << 32), -1)])
def test_layer_norm_rejects(L, change, status):
    assert _norm(L, **change) == status
    assert _norm_back(L, **change) == status


def test_layer_norm_rejects_one_way(L):
    assert _norm(L, y=None) == -1
    assert _norm(L, eps=-1.0) == -1 and _norm(L, eps=float("nan")) == -1
    assert _norm_back(L, dy=None) == -1
    assert _norm_back(L, ws=None) == -3 and _norm_back(L, wsb=16) == -3
    assert _norm(L, N=0, x=None, y=None) == 0               # nothing launched
    assert L.ddm_layer_norm_backward_workspace_bytes(100, 9000, 0) == 0
    assert L.ddm_layer_norm_backward_workspace_bytes(100000, 1024, 2) >= 2 * 1024 * 4


def _loss(L, backward=False, **kw):
    a = dict(g=FAKE, a=FAKE, b=FAKE, la=FAKE, lb=FAKE, cu=FAKE, B=2, P=100, d=24, dtype=1, t=0.07, loss=FAKE, da=FAKE, db=FAKE,
             ws=FAKE, wsb=BIG)
    a.update(kw)
    view = lambda *n: [a[x] for x in n]  # noqa: E731
    if backward:
        return L.ddm_matching_loss_backward(*view("g", "a", "b", "la", "lb", "cu", "B", "P", "d", "dtype", "t", "da", "db", "ws",
                                                  "wsb"), None)
    return L.ddm_matching_loss_forward(*view("a", "b", "cu", "B", "P", "d", "dtype", "t", "loss", "la", "lb", "ws", "wsb"), None)


@pytest.mark.parametrize("change,status", [(dict(a=None), -1), (dict(b=FAKE + 1), -1), (dict(la=None), -1), (dict(cu=None), -1),
                                           (dict(B=0), -1), (dict(P=-1), -1), (dict(P=(1 << 28) + 1), -1), (dict(d=0), -4),
                                           (dict(d=129), -4), (dict(dtype=9), -4), (dict(t=0.0), -1), (dict(t=-0.1), -1),
                                           (dict(t=float("nan")), -1), (dict(ws=None), -3), (dict(wsb=16), -3)])
def test_matching_loss_rejects(L, change, status):
    assert _loss(L, **change) == status
    assert _loss(L, backward=True, **change) == status


def test_matching_loss_rejects_one_way(L):
    assert _loss(L, loss=None) == -1
    assert _loss(L, backward=True, g=None) == -1 and _loss(L, backward=True, da=None) == -1
    assert _loss(L, P=0, a=None, b=None) == 0
    assert L.ddm_matching_loss_workspace_bytes(1, 100, 129, 1) == 0
    assert L.ddm_matching_loss_workspace_bytes(1, 100, 24, 1) > 0
