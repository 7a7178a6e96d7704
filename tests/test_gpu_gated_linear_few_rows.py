"""Few rows of the gated layer, on both sides of where another kernel takes them over: by rows, by the length of k and by the hidden width.
The bounds are those of the layer's other tests: rounding to the type, u, of h, sums of C + 8 terms in 32 bits and silu's 2^-24 (|g| + 8) 4."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("cols,hidden", [(8192, 40), (4100, 130), (1024, 264), (72, 4200), (513, 700)])
def test_values(dtype, cols, hidden):
    import dense_descriptor_matching_amd as ddm
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, b = r(65, cols).to(dtype), (r(2 * hidden, cols) / math.sqrt(cols)).to(dtype), r(2 * hidden).to(dtype)
    p = x.double() @ w.double().T + b.double()
    err = (cols + 8) * E * (x.double().abs() @ w.double().abs().T) + E * p.abs()
    gate, up, gate_err, up_err = p[:, :hidden], p[:, hidden:], err[:, :hidden], err[:, hidden:]
    a = gate * torch.sigmoid(gate)
    a_err = 1.13 * gate_err + (gate.abs() + 8) * 4 * E * a.abs()
    want = a * up
    tol = (U[dtype] + E) * want.abs() + a_err * up.abs() + a.abs() * up_err + a_err * up_err + (2.0 ** -25 if dtype == torch.float16 else 0)
    for rows in (1, 2, 8, 9, 16, 17, 31, 32, 33, 40, 47, 48, 63, 64, 65):
        h, kept = ddm.gated_linear_forward(x[:rows], w, b, keep=True)
        assert ((h.double() - want[:rows]).abs() <= 1.25 * tol[:rows]).all(), rows
        assert ((kept.double() - p[:rows]).abs() <= 1.25 * (err[:rows] + U[dtype] * p[:rows].abs() + 2.0 ** -25)).all(), rows
        assert torch.equal(ddm.gated_linear_forward(x[:rows], w, b)[0], h)
