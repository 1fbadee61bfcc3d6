"""Batches of paged caches whose tables or starts one sequence has put out of order: the others'
results, in every call over such a cache, are as if it had kept the rules."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from spgemm_irregular_matrices_amd import binding  # noqa: E402
from tests import test_gpu_attention_paths as paths  # noqa: E402
from tests import test_gpu_cache as quantized  # noqa: E402
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


def _sequences(count):
    """Texts of which some are cut, and joined, and most have new tokens."""
    rng = np.random.default_rng(count)
    seqs = [(900, 2), (70, 3), (33, 1), (1200, 2)]
    if count > 4:
        new = rng.integers(0, 3, count)
        seqs = [(int(m + rng.integers(0, 90)), int(m)) for m in new]
        seqs[1], seqs[count // 2], seqs[count - 1] = (900, 3), (700, 2), (1200, 1)
        seqs[count // 2 - 1], seqs[count - 2] = (40, 1), (50, 2)  # (a broken one's NaN rows end within two)
    return seqs


def _starts(seqs, index):
    """(broken starts, sequences that they break, rows that no sequence has then)."""
    start = index["q_rowptr"]
    n = len(seqs)
    for at in sorted({0, 1, 2, n // 2, n - 1}):
        for value in (10 ** 9, -1, 2 ** 62, -2 ** 62):
            bad = {at - 1, at} & set(range(n))
            # the one before it has too many rows or none, the one behind it none
            nan = slice(0, 0)
            if value > 0 and at > 0:
                first = int(start[at - 1])
                nan = slice(first, first + max(m for _, m in seqs))
            rows = np.zeros(int(start[-1]), dtype=bool)
            for s in bad:
                rows[int(start[s]):int(start[s + 1])] = True
            rows[nan] = False
            yield _broken(start, at, value), bad, rows, nan


@pytest.mark.parametrize("count", [4, 100, 300])
@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_latent_starts_out_of_order(form, count):
    seqs = _sequences(count)
    c = _latent_batch(form, seqs)
    for start, bad, rows, nan in _starts(seqs, c):
        out = torch.full((len(c["q"]), 4, 48 if form == "expanded" else 128), 7.0, dtype=BF16, device="cuda")
        lse = torch.full(out.shape[:2], 9.0, device="cuda")
        latents._run(dict(c, q_rowptr=start), out=out, lse=lse)
        latents._check(c, seqs, out, lse, skip=bad)
        assert (out[:len(rows)][rows] == 7).all() and (lse[:len(rows)][rows] == 9).all()
        assert torch.isnan(out[nan]).all() and torch.isnan(lse[nan]).all()


@pytest.mark.parametrize("hq", [2, 16])
@pytest.mark.parametrize("count", [4, 100, 300])
def test_quantized_starts_out_of_order(count, hq):
    """Attention in both kernels; 300 texts are cut in pieces, the others evenly."""
    seqs = _sequences(count)
    rng = np.random.default_rng(52)
    c, index, kept, tokens = quantized._filled(rng, seqs, 64, 2, 16, "e4m3")
    q = quantized._query(rng, tokens, hq, 64, BF16)
    for start, bad, rows, nan in _starts(seqs, index):
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 9.0, device="cuda")
        c.attention(q, **{**index, "q_rowptr": start}, out=out, lse=lse)
        quantized._check(c, index, kept, seqs, q, out, lse, 0.125, skip=bad)
        assert (out[:len(rows)][rows] == 7).all() and (lse[:len(rows)][rows] == 9).all()
        assert torch.isnan(out[nan]).all() and torch.isnan(lse[nan]).all()


@pytest.mark.parametrize("count", [4, 100, 300])
def test_rows_of_intact_sequences_are_stored_and_read(count):
    seqs = _sequences(count)
    rng = np.random.default_rng(53)
    index, pool, order, rowptr, tokens = quantized._index(rng, seqs, 16, 3)
    x = quantized._query(rng, tokens, 2, 64, BF16)
    whole = quantized._empty(pool, 16, 2, 64, "e4m3")
    whole.write(x, -x, **index)
    first = index["q_rowptr"].tolist()
    for start, bad, rows, nan in _starts(seqs, index):
        batch = {**index, "q_rowptr": start}
        c = quantized._empty(pool, 16, 2, 64, "e4m3")
        c.write(x, -x, **batch)
        k, v = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
        whole.read(**batch, k=k, v=v)
        k0, v0 = whole.read(**index, tokens=tokens)
        for s, (n, m) in enumerate(seqs):
            at = np.arange(n - m, n)
            where = (torch.from_numpy(order[rowptr[s] + at // 16]).cuda(), torch.from_numpy(at % 16).cuda())
            for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
                got = getattr(c, name)[where]
                want = torch.full_like(got, 0xa5) if s in bad else getattr(whole, name)[where]
                assert torch.equal(got, want), (s, name)
            if s not in bad:
                mine = slice(first[s], first[s + 1])
                assert torch.equal(k[mine], k0[mine]) and torch.equal(v[mine], v0[mine]), s
        assert (k[:len(rows)][rows] == 7).all() and (v[:len(rows)][rows] == 7).all()
        assert torch.isnan(k[nan]).all() and torch.isnan(v[nan]).all()


@pytest.mark.parametrize("count", [4, 100])
def test_paged_starts_out_of_order(count):
    seqs = _sequences(count)
    c = paths._paged_case(np.random.default_rng(54), BF16, 64, 4, 2, 16, seqs)
    for start, bad, rows, nan in _starts(seqs, c):
        out = torch.full_like(c["q"], 7.0)
        lse = torch.full(out.shape[:2], 9.0, device="cuda")
        paths._paged_run(dict(c, q_rowptr=start), out=out, lse=lse, scale=0.125)
        paths._paged_check(c, seqs, 0.125, out, lse, skip=bad)
        assert (out[:len(rows)][rows] == 7).all() and (lse[:len(rows)][rows] == 9).all()
        assert torch.isnan(out[nan]).all() and torch.isnan(lse[nan]).all()


@pytest.mark.parametrize("form", quantized.FORMS)
def test_tensors_of_one_allocation_are_written(form):
    """Tensors that lie between each other's places, by page, by slot and by head, are apart; the
    same bytes for keys and values are not, and are read."""
    from spgemm_irregular_matrices_amd import cache
    rng = np.random.default_rng(55)
    index, pool, order, rowptr, tokens = quantized._index(rng, [(40, 7), (33, 5)], 16, 0)
    x = quantized._query(rng, tokens, 2, 64, BF16)
    plain = quantized._empty(pool, 16, 2, 64, form)
    plain.write(x, -x, **index)
    want = plain.read(**index, tokens=tokens)
    w = 64 if form == "e4m3" else 32
    for cut in range(4):  # the axis inside which the four lie one after another
        lead, places = (pool, 16, 2)[:cut], (pool, 16, 2)[cut:]
        size = [int(np.prod(places)) * n for n in (w, 2, w, 2)]
        at = np.concatenate([[0], np.cumsum([(n + 15) // 16 * 16 for n in size])])
        room = torch.zeros(*lead, int(at[-1]), dtype=torch.uint8, device="cuda")
        parts = [room[..., a:a + n].unflatten(-1, (*places, -1)) for a, n in zip(at, size)]
        c = cache.QuantizedCache(*parts, form)
        c.write(x, -x, **index)
        got = c.read(**index, tokens=tokens)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    both = cache.QuantizedCache(plain.k_codes, plain.k_scales, plain.k_codes, plain.k_scales, form)
    k, v = both.read(**index, tokens=tokens)
    assert torch.equal(k, want[0]) and torch.equal(v, want[0])
    with pytest.raises(binding.SpgemmError):
        both.write(x, x, **index)


class _WithoutLse:
    """The library, with NULL for a call's lse (its argument before the workspace)."""

    def __init__(self, lib):
        self._lib = lib

    def __getattr__(self, name):
        entry = getattr(self._lib, name)
        if name.endswith("_workspace"):
            return entry
        return lambda *args: entry(*args[:-4], None, *args[-3:])


@pytest.mark.parametrize("seqs", [[(900, 1), (5, 1), (70, 1)], [(900, 40), (5, 5), (130, 64)]])
@pytest.mark.parametrize("call", ["absorbed", "expanded", "quantized"])
def test_results_without_lse(call, seqs, monkeypatch):
    """The log-sum-exps may be left out: the results are the same, whole or joined."""
    from spgemm_irregular_matrices_amd import cache, latent
    if call == "quantized":
        c, index, _, tokens = quantized._filled(np.random.default_rng(56), seqs, 64, 2, 16, "e4m3")
        q = quantized._query(np.random.default_rng(57), tokens, 8, 64, BF16)
        run = lambda **more: c.attention(q, **index, **more)  # noqa: E731
    else:
        c = _latent_batch(call, seqs)
        run = lambda **more: latents._run(c, **more)  # noqa: E731
    want, lse = run()
    for module in (cache, latent):
        monkeypatch.setattr(module, "load", lambda lib=_WithoutLse(module.load()): lib)
    untouched = torch.full_like(lse, 9.0)
    out, _ = run(lse=untouched)
    some = sum(m for _, m in seqs)
    assert torch.equal(out[:some], want[:some]) and (untouched == 9).all()
