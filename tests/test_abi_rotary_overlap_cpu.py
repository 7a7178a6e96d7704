"""Host-side checks of rotary outputs that lie over one another or over inputs that are still read. Addresses are made up; every call
is refused before anything is enqueued."""
import os

import pytest

Q, K, QO, KO = (i << 40 for i in (1, 2, 3, 4))


@pytest.fixture(scope="module")
def L():
    import dense_descriptor_matching_amd as ddm
    if not os.path.exists(ddm.LIB_PATH):
        pytest.fail("libddm.so not built: run __graft_entry__.build()")
    return ddm.lib()


def rotary(L, **kw):
    a = dict(q=Q, qt=256, qh=64, Hq=4, k=K, kt=128, kh=64, Hk=2, pos=1 << 30, freq=1 << 31, T=10, D=64, axes=2, pairs=16, dtype=1,
             interleaved=0, inverse=0, m=1.0, qo=QO, qot=256, qoh=64, ko=KO, kot=128, koh=64)
    a.update(kw)
    return L.ddm_rotary(*a.values(), None)


@pytest.mark.parametrize("change", [
    dict(qo=KO), dict(qo=KO + 126), dict(qo=KO - 126),                                   # the outputs over each other
    dict(qo=K), dict(qo=K - 64), dict(ko=Q), dict(ko=Q + 64), dict(qo=K, ko=Q),          # one over the other's input
    dict(qo=Q + 2), dict(qo=Q - 2), dict(ko=K + 126),                                    # over its own input, shifted
    dict(qo=Q, qot=512), dict(qo=Q, qoh=128, qot=256 * 4), dict(ko=K, kot=64, koh=640),  # over its own input, in another order
    dict(qot=63), dict(qot=0), dict(qoh=63), dict(koh=1), dict(qot=64), dict(kot=64, koh=64), dict(kot=192, koh=160)])
def test_overlaps_are_refused(L, change):
    assert rotary(L, **change) == -1


@pytest.mark.parametrize("change,status", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1), (dict(ko=None), -1), (dict(q=Q + 1), -1), (dict(ko=KO + 1), -1),
    (dict(pos=None), -1), (dict(pos=(1 << 30) + 2), -1), (dict(freq=None), -1), (dict(freq=(1 << 31) + 4), -1), (dict(T=-1), -1),
    (dict(D=63), -1), (dict(axes=0), -1), (dict(pairs=0), -1), (dict(pairs=17), -1), (dict(axes=3), -1), (dict(interleaved=2), -1),
    (dict(inverse=-1), -1), (dict(m=float("nan")), -1), (dict(m=1e39), -1), (dict(Hq=-1), -1), (dict(Hk=65537), -1), (dict(qt=-1), -1),
    (dict(koh=-64), -1), (dict(kt=1 << 41), -1)])
def test_other_refusals_without_overlaps(L, change, status):
    assert rotary(L, **change) == status
