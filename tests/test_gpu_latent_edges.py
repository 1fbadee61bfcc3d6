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


def _wild_columns(c, clean, got, seqs, seen_from, columns, head=None):
    """The first sequence's rows from seen_from on have these values in these columns (of one head)
    and are else within the bounds of the clean ones; all other rows are the clean ones."""
    new = seqs[0][1]
    rows = slice(seen_from, new)
    heads = range(c["q"].shape[1])
    for h in heads:
        for m, value in columns.items():
            if head is None or h == head:
                x = f64(got[0][rows, h, m])
                assert (np.isnan(x) if np.isnan(value) else x == value).all(), (h, m, x)
                got[0][rows, h, m] = clean[0][rows, h, m]
    assert torch.equal(got[0][:seen_from], clean[0][:seen_from]) and torch.equal(got[1][:seen_from], clean[1][:seen_from])
    some = sum(m for _, m in seqs)
    assert torch.equal(got[0][new:some], clean[0][new:some]) and torch.equal(got[1][new:some], clean[1][new:some])
    latents._check(c, seqs, *got)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("heads,new,dv", [(3, 40, 48), (48, 300, 128)])
def test_infinite_made_values_reach_their_columns_alone(heads, new, dv, dtype):
    """Values past the type's range in some columns of one head, of keys that all rows of a tile see
    and of such that only later ones do: infinite there, and NaN where two signs meet."""
    rng = np.random.default_rng(61)
    # (of 48 heads in tiles of 256 rows)
    seqs = [(400 + new, new), *([(300, 300), (257, 257)] if new == 300 else [(31, 7)])]
    c = latents._case(rng, dtype, seqs, heads, 128, 32, 16, 64, dv, pad=0)
    # what latents hold in place 7 gets to no key, and only in one head to two columns
    for w in c["w"]:
        w[:, :, 7] = 0
    for s, (n, _) in enumerate(seqs):
        c["kept"][s][:, 7] = 0
        page = c["table"].col[int(c["table"].rowptr[s]):int(c["table"].rowptr[s + 1])].long()
        c["cache"][page, :, 7] = 0
    big = {BF16: 2.0 ** 100, F16: 2.0 ** 15}[dtype]
    clean = latents._run(c)
    latents._check(c, seqs, *clean)
    one = c["w"][1][1].clone()
    c["w"][1][1, 2, 7], c["w"][1][1, dv - 1, 7] = big, -big
    inf = float("inf")
    for token in (0, 390, 400, 400 + new // 2, 400 + new - 1):
        _put(c, token, {7: big})
        got = [x.clone() for x in latents._run(c)]
        c["w"][1][1], whole = one, c["w"][1][1].clone()  # (the bounds' values are the clean ones)
        _wild_columns(c, clean, got, seqs, max(0, token - 400), {2: inf, dv - 1: -inf}, head=1)
        c["w"][1][1] = whole
        if token >= 400:  # another one, of the other sign, that all rows see
            _put(c, 60, {7: -big})
            got = [x.clone() for x in latents._run(c)]
            x = f64(got[0][:new, 1, 2])
            assert np.isnan(x[token - 400:]).all() and (x[:token - 400] == -inf).all()
            x = f64(got[0][:new, 1, dv - 1])
            assert np.isnan(x[token - 400:]).all() and (x[:token - 400] == inf).all()
            _put(c, 60, {7: 0.0})
        _put(c, token, {7: 0.0})


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("scale", [0.1, -0.1])
@pytest.mark.parametrize("new", [3, 40])
def test_an_infinite_value_of_weight_0(new, scale, dtype, form):
    """A key whose score is -infinity has no weight, and 0 times its infinite value is NaN: in that
    value's column, wherever the key lies, and in no other, whose results do not know the key."""
    rng = np.random.default_rng(62)
    seqs = [(400 + new, new), (31, min(new, 7))]
    c = latents._case(rng, dtype, seqs, 3, 128, 32, 16, pad=0, **(dict(dn=64, dv=48) if form == "expanded" else {}))
    column = 7
    for s, (n, _) in enumerate(seqs):
        c["kept"][s][:, 7] = 0
        page = c["table"].col[int(c["table"].rowptr[s]):int(c["table"].rowptr[s + 1])].long()
        c["cache"][page, :, 7] = 0
    c["q"][:, :, 7] = -1.0 if scale > 0 else 1.0
    value = float("inf")
    if form == "expanded":  # one value of the keys and one of the values are infinite
        big = {BF16: 2.0 ** 100, F16: 2.0 ** 15}[dtype]
        value, column = big, 5
        for w in c["w"]:
            w[:, :, 7] = 0
        c["w"][0][:, 7, 7] = c["w"][1][:, 5, 7] = big
    c["scale"] = scale
    clean = latents._run(c)
    latents._check(c, seqs, *clean)
    for token in (0, 390, 400, 400 + new - 1):
        page = int(c["table"].col[token // 16])
        old = c["cache"][page, token % 16].clone()
        c["cache"][page, token % 16, 7] = value
        out, lse = latents._run(c)
        # the same without the key, by a score that leaves it no weight either
        c["cache"][page, token % 16] = 0
        c["cache"][page, token % 16, 7] = 2.0 ** 14
        if form == "expanded":
            c["w"][1][:, 5, 7] = 0
        want, wlse = latents._run(c)
        if form == "expanded":
            c["w"][1][:, 5, 7] = big
        c["cache"][page, token % 16] = old
        first = max(0, token - 400)
        assert torch.isnan(out[first:new, :, column]).all(), token
        out[first:new, :, column] = want[first:new, :, column]
        assert torch.equal(out[first:new], want[first:new]) and torch.equal(lse[first:new], wlse[first:new]), token
        assert torch.equal(out[:first], clean[0][:first]) and torch.equal(lse[:first], clean[1][:first])
        assert torch.equal(out[new:], clean[0][new:]) and torch.equal(lse[new:], clean[1][new:])


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_expanded_in_groups_of_heads(dtype):
    """A call's workspace is for all of its heads: groups of them, as slices, need a part of it and
    give their results."""
    from spgemm_irregular_matrices_amd import latent
    seqs = [(300, 40), (1, 1), (700, 65)]
    c = latents._case(np.random.default_rng(63), dtype, seqs, 6, 128, 32, 16, 64, 48, pad=2)
    index = dict(pages=c["table"], q_rowptr=c["q_rowptr"], lengths=c["lengths"], max_q=c["max_q"], max_len=c["max_len"])
    out = torch.full((len(c["q"]), 6, 48), 7.0, dtype=dtype, device="cuda")
    lse = []
    for h in (slice(0, 2), slice(2, 3), slice(3, 6)):
        _, part = latent.latent_attention_expanded(c["q"][:, h], c["cache"], c["w"][0][h], c["w"][1][h], **index,
                                                   scale=c["scale"], out=out[:, h])
        lse.append(part)
    latents._check(c, seqs, out, torch.cat(lse, 1))
    assert (out[-2:] == 7).all()


@pytest.mark.parametrize("count,heads,new", [(256, 128, 1), (300, 128, 1), (1024, 16, 1), (1025, 16, 1), (64, 128, 4), (90, 40, 5)])
def test_a_long_text_among_many(count, heads, new):
    """Cut evenly over the card, with those around it, up to 1024 texts; with one that breaks the
    rules. Every call gives the same bits."""
    rng = np.random.default_rng(count)
    seqs = [(int(n) + new, new) for n in rng.integers(0, 60, count)]
    seqs[count // 3], seqs[count - 1] = (2500, new), (700, min(2, new))
    c = latents._case(rng, BF16, seqs, heads, 64, 16, 16, pad=1)
    out, lse = latents._run(c)
    latents._check(c, seqs, out, lse)
    again = latents._run(c)
    some = sum(m for _, m in seqs)
    assert torch.equal(out[:some], again[0][:some]) and torch.equal(lse[:some], again[1][:some])
    c["lengths"][count // 2] = 10 ** 6
    out, lse = latents._run(c)
    latents._check(c, seqs, out, lse, skip=(count // 2,))
    start = int(c["q_rowptr"][count // 2])
    assert torch.isnan(out[start:start + new]).all() and torch.isnan(lse[start:start + new]).all()
