"""Row strides of the gated layer end at 4 MB; those whose bytes would not fit into 64 bits are beyond that too. Host checks alone."""
import os

import pytest

FAKE = 1 << 40        # 16-byte aligned, never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def L():
    import dense_descriptor_matching_amd as ddm
    if not os.path.exists(ddm.LIB_PATH):
        pytest.fail("libddm.so not built: run __graft_entry__.build()")
    return ddm.lib()


@pytest.mark.parametrize("dtype,bytes_", [(0, 4), (1, 2), (2, 2)])
@pytest.mark.parametrize("ldx", [(1 << 62) + 64, 1 << 62, (1 << 63) - 1, (1 << 61) + 64, 1 << 32, None])
def test_strides_beyond_4_mb(L, ldx, dtype, bytes_):
    ldx = (1 << 22) // bytes_ + 1 if ldx is None else ldx
    assert L.ddm_gated_linear_forward(FAKE, ldx, FAKE, FAKE, 100, 64, 48, dtype, 0, FAKE, FAKE, FAKE, 1 << 50, None) == -1
    assert L.ddm_gated_linear_backward(FAKE, FAKE, ldx, FAKE, FAKE, 100, 64, 48, dtype, 0, FAKE, FAKE, FAKE, FAKE, 1 << 50, None) == -1
