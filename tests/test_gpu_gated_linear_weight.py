"""Where the gated layer's weight may begin: on any element if its rows are not whole 16-byte pieces, as they are repacked; else on a
16-byte boundary."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ddm():
    import dense_descriptor_matching_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [3, 50, 200])
@pytest.mark.parametrize("cols", [1, 61, 131])
def test_parameters_in_one_flat_buffer(ddm, dtype, rows, cols):
    hidden = 37
    flat = torch.randn(2 * hidden * (cols + 1) + 1, device="cuda").div_(math.sqrt(cols)).to(dtype)
    x, dh = torch.randn(rows, cols, device="cuda").to(dtype), torch.randn(rows, hidden, device="cuda").to(dtype)
    w, b = flat[1:1 + 2 * hidden * cols].view(2 * hidden, cols), flat[1 + 2 * hidden * cols:]
    assert w.data_ptr() % 16 and w.is_contiguous()

    def step(w, b):
        h, kept = ddm.gated_linear_forward(x, w, b, keep=True)
        return (h,) + ddm.gated_linear_backward(dh, x, w, kept)

    got, want = step(w, b), step(w.clone(), b.clone())
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_rows_of_whole_pieces(ddm):
    x = torch.randn(4, 32, device="cuda").half()
    w = torch.randn(20 * 32 + 4, device="cuda").half()[4:].view(20, 32)
    with pytest.raises(ddm.DDMError, match="16-byte boundary") as e:
        ddm.gated_linear_forward(x, w)
    assert e.value.status == -1
    h, kept = ddm.gated_linear_forward(x, w.clone(), keep=True)
    with pytest.raises(ddm.DDMError, match="16-byte boundary"):
        ddm.gated_linear_backward(h, x, w, kept)
    _, dw, db = ddm.gated_linear_backward(h, x, w, kept, need_dx=False)          # the weight is not read
    _, want, wb = ddm.gated_linear_backward(h, x, w.clone(), kept)
    assert torch.equal(dw, want) and torch.equal(db, wb)
