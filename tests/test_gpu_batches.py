"""Batches of paged caches whose tables or starts one sequence has put out of order: the others'
results, in every call over such a cache, are as if it had kept the rules."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from spgemm_irregular_matrices_amd import binding  # noqa: E402
from tests import test_gpu_latent as latents  # noqa: E402

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from spgemm_irregular_matrices_amd import cache, latent
    cache.load()
    latent.load()


def _broken(values, at, value):
    values = values.clone()
    values[at] = value
    return values


def _latent_batch(form, seqs, **more):
    extra = dict(dn=64, dv=48) if form == "expanded" else {}
    return latents._case(np.random.default_rng(50), BF16, seqs, 4, 128, 32, 16, **extra, **more)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("many", [False, True])
def test_latent_tables_out_of_order(form, many):
    """The table's row pointers of two neighbouring sequences are broken."""
    seqs = [(40, 2), (70, 3), (33, 1), (20, 2)]
    if many:
        seqs = [(int(n), min(int(n), 2)) for n in np.random.default_rng(51).integers(1, 90, 150)]
    c = _latent_batch(form, seqs)
    latents._check(c, seqs, *latents._run(c))
    t = c["table"]
    for at in (1, 2, len(seqs) - 1):
        for value in (10 ** 9, -1, 2 ** 62, 0):
            # what an earlier call left in the workspace is no one's keys
            latents._run(dict(c, cache=torch.full_like(c["cache"], float("nan"))))
            table = binding.DeviceCSR(t.nrows, t.ncols, _broken(t.rowptr, at, value), t.col, None)
            got = latents._run(dict(c, table=table))
            # with 0 the second one keeps the rules, with other pages than its own
            latents._check(c, seqs, *got, skip=(at - 1, at))
            first = sum(m for _, m in seqs[:at - 1])
            assert torch.isnan(got[0][first:first + seqs[at - 1][1]]).all()
