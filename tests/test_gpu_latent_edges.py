"""Latent attention where scores or values are at the edge of what a type holds, in both forms."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import test_gpu_latent as latents  # noqa: E402
from tests.attention_ref import f64  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from spgemm_irregular_matrices_amd import latent
    latent.load()


def _put(c, token, values):
    """Values of a token of the first sequence, whose pages have 16 slots."""
    page = int(c["table"].col[token // 16])
    for x, value in values.items():
        c["cache"][page, token % 16, x] = value
        c["kept"][0][token, x] = float(c["cache"][page, token % 16, x])


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("heads,new", [(2, 1), (2, 40), (128, 1)])
def test_scores_in_steps_past_the_slack(dtype, odd, heads, new, form):
    """Scores of 2^27 in base 2, whose steps in floats are 16: the next larger one is 2^16 times
    the weight, wherever the reference's place among the steps rounds a smaller sum to."""
    rng = np.random.default_rng(60)
    n = 200
    c = latents._case(rng, dtype, [(n, new)], heads, 64, 0, 16, pad=0,
                      **(dict(dn=16, dv=32) if form == "expanded" else {}))
    c["scale"] = float(np.log(2.0))  # the factor of scores in base 2 is 1
    for j in range(n):  # scores, exact in floats: 2^27 + 16 (odd + 1), from token 100 on 16 more
        _put(c, j, {0: 2.0 ** 14, 1: 1.0 + odd + (j >= 100)})
    c["q"][:] = 0
    c["q"][:, :, 0], c["q"][:, :, 1] = 2.0 ** 13, 16.0
    if "w" in c:
        c["w"][0][:] = 0  # keys' first two values are the latents'
        c["w"][0][:, 0, 0] = c["w"][0][:, 1, 1] = 1.0
    out, lse = latents._run(c)
    x = c["kept"][0]
    v, err = np.repeat(x[:, None], heads, 1), 0.0
    if "w" in c:
        v, err = latents._made(x, c["w"][1], dtype)
    u = {BF16: 2.0 ** -8, F16: 2.0 ** -11}[dtype]
    for t in range(new):
        sees = n - new + t + 1
        w = np.where(np.arange(n) >= 100, 1.0, 2.0 ** -16)[:sees]  # exact in both types
        total = w.sum()
        want = np.tensordot(w / total, v[:sees], (0, 0))
        # one rounding of a result; sums of up to 200 products in floats; the made values'
        bound = u * np.abs(want) + 2.0 ** -15 * np.tensordot(w / total, np.abs(v[:sees]), (0, 0))
        bound = bound + np.tensordot(w / total, err[:sees], (0, 0)) if "w" in c else bound
        got = f64(out[t])
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= bound + 2.0 ** -25).all()
        # two sums of 2^27 in base 2, to 8 each; ln 2 to 2^-25 of it; the result to 4
        assert (np.abs(f64(lse[t]) - (2.0 ** 27 + 16 * (odd + 2)) * np.log(2.0) - np.log(total)) <= 20).all()
