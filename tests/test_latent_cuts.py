"""Absorbed latent attention cuts the keys of batches of any size that it is made for (CPU: a call
whose keys are not cut needs no workspace)."""
import pytest

torch = pytest.importorskip("torch")

from spgemm_irregular_matrices_amd import latent  # noqa: E402
from tests.test_cache_abi import _latent_bytes  # noqa: E402


@pytest.mark.parametrize("heads", [1, 20, 128])
@pytest.mark.parametrize("seqs,new", [(1, 1), (2, 30), (64, 1), (64, 4), (128, 2), (255, 1), (256, 1), (257, 1), (300, 2),
                                      (1000, 1), (1024, 1)])
def test_long_texts_are_cut(heads, seqs, new):
    d = latent.LatentDesc(0, heads, 512, 64, 0, 0, 0.1)
    rc, n = _latent_bytes(d, seqs=seqs, tokens=seqs * new, max_new=new, max_length=32768)
    # two parts a range and row of a tile, 512 values and two more each
    assert rc == 0 and 0 < n <= 2 * 256 * 128 * 514 * 4 + 512
    assert _latent_bytes(d, seqs=seqs, tokens=seqs * new, max_new=new, max_length=64) == (0, 0)


def test_batches_of_mostly_empty_tiles_are_not_cut_further():
    """One long chunk beside many single tokens: its tiles would be everyone's."""
    d = latent.LatentDesc(0, 128, 512, 64, 0, 0, 0.1)
    assert _latent_bytes(d, seqs=1000, tokens=1029, max_new=30, max_length=32768) == (0, 0)
