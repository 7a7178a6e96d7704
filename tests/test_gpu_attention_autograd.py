"""What autograd hands to attention's gradient."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import ddm, make, run  # noqa: E402,F401  (ddm is a fixture)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_gradient_off_a_16_byte_boundary(ddm, dtype):
    """Autograd hands on views: joined behind one other element, the gradient of out begins at an odd element."""
    x = make(dtype, 4, 2, 64, (70, 33), (70, 33), seed=41)
    want = run(ddm, x, True, 64 ** -0.5)
    q, k, v = (x[n].clone().requires_grad_() for n in ("q", "k", "v"))
    one = torch.zeros(1, dtype=q.dtype, device="cuda", requires_grad=True)
    joined = torch.cat([one, ddm.attention(q, k, v, x["cu_q"], x["cu_k"], causal=True).flatten()])
    joined.backward(torch.cat([x["dout"].new_zeros(1), x["dout"].flatten()]))
    for t, n in ((q, "dq"), (k, "dk"), (v, "dv")):
        assert torch.equal(t.grad, want[n]), n
