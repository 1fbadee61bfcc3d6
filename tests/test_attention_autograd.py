"""Attention calls are not recorded by autograd, and say so (CPU: refused before any GPU work)."""
import pytest

torch = pytest.importorskip("torch")

from spgemm_irregular_matrices_amd import attention, binding  # noqa: E402


class _Plan(attention.AttentionPlan):
    """A plan's checks without a plan."""

    def __init__(self):
        self._h, self.device = None, torch.device("cpu")
        self.nrows = self.ncols = 2


def _tensors(grad):
    return [torch.zeros(2, 1, 64, requires_grad=i == grad) for i in range(5)]


@pytest.mark.parametrize("grad", range(3))
def test_inputs_that_require_gradients_are_refused(grad):
    q, k, v, out, dout = _tensors(grad)
    with pytest.raises(ValueError, match="autograd"):
        _Plan().forward(q, k, v)
    with pytest.raises(ValueError, match="autograd"):
        _Plan().backward(dout, q, k, v, out, torch.zeros(2, 1))
    with pytest.raises(ValueError, match="closed"):  # fine without recording: the next check
        with torch.no_grad():
            _Plan().forward(q, k, v)
    table = binding.DeviceCSR(1, 2, torch.tensor([0, 1]), torch.zeros(1, dtype=torch.int32), None)
    cache = [torch.zeros(2, 16, 1, 64, requires_grad=i == grad) for i in range(1, 3)]
    call = lambda: attention.paged_attention(q, *cache, table, torch.tensor([0, 2]),  # noqa: E731
                                             torch.tensor([2]), 2, 2)
    with pytest.raises(ValueError, match="autograd"):
        call()
    with torch.inference_mode(), pytest.raises(ValueError, match="on the GPU"):
        call()


@pytest.mark.parametrize("grad", range(3, 5))
def test_what_the_gradients_take_is_refused_too(grad):
    q, k, v, out, dout = _tensors(grad)
    with pytest.raises(ValueError, match="autograd"):
        _Plan().backward(dout, q, k, v, out, torch.zeros(2, 1))


def test_inside_a_function_of_autograd():
    """Where a user's own Function calls, nothing is recorded and nothing refused."""
    q, k, v, _, _ = _tensors(0)

    class Function(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v):
            return _Plan().forward(q, k, v)[0]

    with pytest.raises(ValueError, match="closed"):
        Function.apply(q, k, v)
