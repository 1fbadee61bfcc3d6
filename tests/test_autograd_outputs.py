"""Calls over masks and caches are refused for what autograd would lose: outputs that require
gradients, and tensors with a tangent in forward mode (CPU: before any GPU work)."""
import pytest

torch = pytest.importorskip("torch")

from torch.autograd import forward_ad  # noqa: E402

from spgemm_irregular_matrices_amd import attention, binding, cache, latent  # noqa: E402
from tests.test_attention_autograd import _Plan  # noqa: E402
from tests.test_cache_abi import _cache  # noqa: E402

TABLE = binding.DeviceCSR(1, 3, torch.tensor([0, 1]), torch.zeros(1, dtype=torch.int32), None)
INDEX = (TABLE, torch.tensor([0, 1]), torch.tensor([1]), 1, 1)
ZEROS = torch.zeros
BF16 = dict(dtype=torch.bfloat16)

# name: (the call of its tensors, the tensors by name, which of them are outputs, what it says on the CPU)
CALLS = {
    "forward": (lambda t: _Plan().forward(t["q"], t["k"], t["v"], out=t["out"], lse=t["lse"]),
                dict(q=(2, 1, 64), k=(2, 1, 64), v=(2, 1, 64), out=(2, 1, 64), lse=(2, 1)), ("out", "lse"), "closed"),
    "backward": (lambda t: _Plan().backward(t["dout"], t["q"], t["k"], t["v"], t["out"], t["lse"], dq=t["dq"],
                                            dk=t["dk"], dv=t["dv"]),
                 dict(q=(2, 1, 64), k=(2, 1, 64), v=(2, 1, 64), out=(2, 1, 64), lse=(2, 1), dout=(2, 1, 64),
                      dq=(2, 1, 64), dk=(2, 1, 64), dv=(2, 1, 64)), ("dq", "dk", "dv"), "closed"),
    "paged": (lambda t: attention.paged_attention(t["q"], t["k"], t["v"], *INDEX, out=t["out"], lse=t["lse"]),
              dict(q=(1, 2, 64), k=(3, 16, 2, 64), v=(3, 16, 2, 64), out=(1, 2, 64), lse=(1, 2)), ("out", "lse"),
              "on the GPU"),
    "write": (lambda t: _cache().write(t["k"], t["v"], *INDEX), dict(k=(1, 2, 64), v=(1, 2, 64)), (), "on the GPU"),
    "read": (lambda t: _cache().read(*INDEX, k=t["k"], v=t["v"]), dict(k=(1, 2, 64), v=(1, 2, 64)), ("k", "v"),
             "on the GPU"),
    "quantized": (lambda t: _cache().attention(t["q"], *INDEX, out=t["out"], lse=t["lse"]),
                  dict(q=(1, 4, 64), out=(1, 4, 64), lse=(1, 4)), ("out", "lse"), "on the GPU"),
    "latent": (lambda t: latent.latent_attention(t["q"], t["c"], *INDEX, value_dim=64, scale=0.1, out=t["out"],
                                                 lse=t["lse"]),
               dict(q=(1, 4, 80), c=(3, 16, 80), out=(1, 4, 64), lse=(1, 4)), ("out", "lse"), "on the GPU"),
    "expanded": (lambda t: latent.latent_attention_expanded(t["q"], t["c"], t["wk"], t["wv"], *INDEX, out=t["out"],
                                                            lse=t["lse"]),
                 dict(q=(1, 4, 48), c=(3, 16, 80), wk=(4, 32, 64), wv=(4, 48, 64), out=(1, 4, 48), lse=(1, 4)),
                 ("out", "lse"), "on the GPU"),
}
EACH = [(name, t) for name, call in CALLS.items() for t in call[1]]


def _tensors(name):
    kind = BF16 if name in ("latent", "expanded") else {}
    return {n: ZEROS(*shape, **({} if n == "lse" else kind)) for n, shape in CALLS[name][1].items()}


@pytest.mark.parametrize("name", CALLS)
def test_calls_get_as_far_as_the_gpu(name):
    call, _, _, says = CALLS[name]
    with pytest.raises(ValueError, match=says):
        call(_tensors(name))
    with forward_ad.dual_level(), pytest.raises(ValueError, match=says):  # a level alone is nothing
        call(_tensors(name))


@pytest.mark.parametrize("name,which", EACH)
def test_tensors_that_require_gradients(name, which):
    call, _, _, says = CALLS[name]
    t = _tensors(name)
    t[which].requires_grad_(True)
    with pytest.raises(ValueError, match="autograd"):
        call(t)
    with torch.no_grad(), pytest.raises(ValueError, match=says):
        call(t)


@pytest.mark.parametrize("name,which", EACH)
def test_tensors_with_a_tangent(name, which):
    call, _, _, says = CALLS[name]
    t = _tensors(name)
    with forward_ad.dual_level():
        t[which] = forward_ad.make_dual(t[which], torch.ones_like(t[which]))
        with pytest.raises(ValueError, match="forward mode"):
            call(t)
        with torch.no_grad(), pytest.raises(ValueError, match="forward mode"):  # (which goes on there)
            call(t)
        t[which] = forward_ad.unpack_dual(t[which]).primal
        with pytest.raises(ValueError, match=says):
            call(t)


def test_inside_a_function_with_a_jvp():
    class Function(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v):
            return CALLS["paged"][0](dict(q=q, k=k, v=v, out=None, lse=None))[0]

    t = _tensors("paged")
    with forward_ad.dual_level(), pytest.raises(ValueError, match="on the GPU"):
        Function.apply(forward_ad.make_dual(t["q"], t["q"]), t["k"], t["v"])
