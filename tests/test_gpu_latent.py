"""Attention over a paged cache of latent vectors on the GPU, in both forms,
through the public calls, against the definition in 64 bits with a bound per
element."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from spgemm_irregular_matrices_amd import binding  # noqa: E402
from tests import attention_ref as ref  # noqa: E402
from tests import cache_ref as cref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
SEQS = [(1, 1), (33, 1), (40, 7), (5, 5), (0, 0), (130, 2), (200, 33), (64, 64)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from spgemm_irregular_matrices_amd import latent
    latent.load()


def _api():
    from spgemm_irregular_matrices_amd import latent
    return latent


def _case(rng, dtype, seqs, heads, dl, dr, page, dn=None, dv=None, pad=3, layout="rows", room=0, size=1.0):
    """A cache with random rows in every sequence's places and NaN in all others.
    dn, dv: the expanded form's widths; room: unused entries of the page table."""
    count = [(n + page - 1) // page for n, _ in seqs]
    pool = sum(count) + 2
    order = rng.permutation(pool)[:sum(count)]
    rowptr = np.concatenate([[0], np.cumsum(count)]).astype(np.int64)
    start = np.concatenate([[0], np.cumsum([m for _, m in seqs])]).astype(np.int64)
    tokens = int(start[-1]) + pad
    rows = torch.full((pool, page, dl + dr), float("nan"), dtype=dtype)
    kept = []
    for s, (n, _) in enumerate(seqs):
        x = torch.from_numpy(rng.standard_normal((n, dl + dr))).to(dtype)
        at = np.arange(n)
        rows[order[rowptr[s] + at // page], at % page] = x
        kept.append(ref.f64(x))
    rows = rows.cuda()
    if layout == "gaps":
        wide = torch.full((pool, page + 1, dl + dr + 24), float("nan"), dtype=dtype, device="cuda")
        wide[:, :page, 8:8 + dl + dr] = rows
        rows = wide[:, :page, 8:8 + dl + dr]
    col = np.concatenate([order, np.full(room, -5)]).astype(np.int32)
    c = dict(table=binding.DeviceCSR(len(seqs), pool, torch.from_numpy(rowptr).cuda(), torch.from_numpy(col).cuda(), None),
             q_rowptr=torch.from_numpy(start).cuda(), lengths=torch.tensor([n for n, _ in seqs], dtype=torch.int64).cuda(),
             max_q=max(m for _, m in seqs), max_len=max(n for n, _ in seqs), cache=rows, kept=kept, dl=dl, dr=dr,
             scale=(dl + dr) ** -0.5)
    width = dl + dr
    if dn:
        width = dn + dr
        c["w"] = [torch.from_numpy(rng.standard_normal((heads, w, dl)) * dl ** -0.5).to(dtype).cuda() for w in (dn, dv)]
        c["scale"] = width ** -0.5
    c["q"] = torch.from_numpy(size * rng.standard_normal((tokens, heads, width))).to(dtype).cuda()
    return c


def _run(c, **more):
    index = dict(pages=c["table"], q_rowptr=c["q_rowptr"], lengths=c["lengths"], max_q=c["max_q"], max_len=c["max_len"])
    if "w" in c:
        return _api().latent_attention_expanded(c["q"], c["cache"], *c["w"], **index, **{"scale": c["scale"], **more})
    return _api().latent_attention(c["q"], c["cache"], **index, value_dim=c["dl"], **{"scale": c["scale"], **more})


# A made key or value: dl products and sums in floats; then rounded to two numbers
# of the type, which leave 2^-16 (bfloat16) or 2^-22 (half, absolutely 2^-25 below its
# normal range) of it.
MADE = {BF16: 2.0 ** -16, F16: 2.0 ** -22}


def _made(x, w, dtype):
    """Keys or values [n, heads, width] of latents x and weights w, and the error of each."""
    w = ref.f64(w)
    y = np.einsum("nx,hmx->nhm", x, w)
    err = (x.shape[1] + 2) * cref.E * np.einsum("nx,hmx->nhm", np.abs(x), np.abs(w)) + MADE[dtype] * np.abs(y)
    return y, err + (2.0 ** -25 if dtype == F16 else 0.0)


def _check(c, seqs, out, lse, skip=(), scale=None):
    """Weights are held relative to a reference within 2^8 of the largest: in half
    precision, whose smallest step is 2^-24 and which holds them times 2^7, that
    loses 2^-32 of the reference's weight."""
    dtype, dl = c["q"].dtype, c["dl"]
    scale = c["scale"] if scale is None else scale
    weight = {BF16: 2.0 ** -8, F16: 2.0 ** -11}[dtype]
    at = 0
    for s, (n, m) in enumerate(seqs):
        if m and s not in skip:
            x = c["kept"][s]
            ke = ve = 0.0
            if "w" in c:
                (k, ke), (v, ve) = _made(x[:, :dl], c["w"][0], dtype), _made(x[:, :dl], c["w"][1], dtype)
                rope = np.broadcast_to(x[:, None, dl:], (n, k.shape[1], c["dr"]))
                k, ke = np.concatenate((k, rope), 2), np.concatenate((ke, 0 * rope), 2)
            else:
                k, v = x[:, None], x[:, None, :dl]
            terms = k.shape[2] * (2 if "w" in c else 1)
            o, l, oe, le = cref.attend(ref.f64(c["q"][at:at + m]), k, v, n - m, scale, dtype, terms, weight,
                                       2 if "w" in c else 1, ke, ve)
            if dtype == F16:
                oe = oe + 2.0 ** -32 * np.abs(v).sum(0).max(0)
            ref.check(out[at:at + m], o, oe, f"out of sequence {s}")
            ref.check(lse[at:at + m], l, le, f"lse of sequence {s}")
        at += m


ABSORBED = [(BF16, 128, 512, 64, 16), (F16, 16, 512, 64, 64), (BF16, 20, 256, 32, 24), (F16, 1, 128, 64, 1),
            (BF16, 7, 96, 0, 5), (BF16, 3, 384, 40, 7), (F16, 33, 224, 8, 128), (BF16, 64, 32, 16, 3)]
EXPANDED = [(BF16, 4, 512, 64, 16, 128, 128), (F16, 3, 256, 32, 7, 64, 64), (BF16, 1, 128, 0, 1, 48, 16),
            (F16, 5, 96, 8, 24, 128, 32), (BF16, 2, 320, 40, 5, 16, 112), (F16, 9, 32, 64, 64, 80, 96)]


@pytest.mark.parametrize("dtype,heads,dl,dr,page", ABSORBED)
def test_absorbed(dtype, heads, dl, dr, page):
    rng = np.random.default_rng(heads * 1000 + page)
    c = _case(rng, dtype, SEQS, heads, dl, dr, page, layout="gaps" if page % 2 else "rows")
    tokens = len(c["q"])
    out = torch.full((tokens, heads, dl), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((tokens, heads), 9.0, device="cuda")
    out, lse = _run(c, out=out, lse=lse)
    _check(c, SEQS, out, lse)
    assert (out[-3:] == 7.0).all() and (lse[-3:] == 9.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("dtype,heads,dl,dr,page,dn,dv", EXPANDED)
@pytest.mark.parametrize("room", [0, 5000])
def test_expanded(dtype, heads, dl, dr, page, dn, dv, room):
    """Also with a page table of much room: made keys then lie by sequence and place."""
    rng = np.random.default_rng(heads * 1000 + page)
    c = _case(rng, dtype, SEQS, heads, dl, dr, page, dn, dv, layout="gaps" if page % 2 else "rows", room=room)
    tokens = len(c["q"])
    out = torch.full((tokens, heads, dv), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((tokens, heads), 9.0, device="cuda")
    out, lse = _run(c, out=out, lse=lse)
    _check(c, SEQS, out, lse)
    assert (out[-3:] == 7.0).all() and (lse[-3:] == 9.0).all()


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("heads,dl,dr", [(128, 512, 64), (16, 256, 64), (5, 128, 32)])
def test_single_tokens(heads, dl, dr, dtype):
    """The next token of sequences of one to 1300 cached ones, pieces joined."""
    rng = np.random.default_rng(31)
    seqs = [(n, 1) for n in (1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 1300)]
    c = _case(rng, dtype, seqs, heads, dl, dr, 16)
    _check(c, seqs, *_run(c))


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("new", [3, 40, 150])
@pytest.mark.parametrize("dl", [512, 128])
def test_chunks_and_wild_tokens(dl, new, dtype, form):
    """Chunks of several tiles; then NaN and infinities in one token that only later
    ones see, in its latent part, in its last part, and with one value only."""
    rng = np.random.default_rng(new)
    seqs = [(340 + new, new), (new, new), (310, max(1, new // 3)), (3, 1)]
    extra = dict(dn=64, dv=64) if form == "expanded" else {}
    c = _case(rng, dtype, seqs, 3, dl, 64, 16, **extra)
    clean = _run(c)
    _check(c, seqs, *clean)
    at = 340 + new // 2
    page = int(c["table"].col[at // 16])
    sees = torch.zeros(len(c["q"]), dtype=torch.bool, device="cuda")
    sees[new // 2:new] = True
    some = sum(m for _, m in seqs)
    row = c["cache"][page, at % 16].clone()
    for where, value in ((slice(None), float("nan")), (slice(dl, None), float("nan")), (slice(5, 6), float("inf")),
                         (slice(dl - 1, dl), -float("inf"))):
        c["cache"][page, at % 16] = row
        c["cache"][page, at % 16, where] = value
        got = _run(c)
        for a, b in zip(got, clean):
            assert torch.equal(a[:some][~sees[:some]], b[:some][~sees[:some]])
        assert not torch.isfinite(got[0][sees].float()).all(-1).any()


@pytest.mark.parametrize("dtype,dl,dr,dn,dv", [(BF16, 128, 64, 128, 128), (F16, 96, 32, 64, 48), (F16, 64, 0, 16, 80)])
def test_long_chunks_of_many_heads(dtype, dl, dr, dn, dv):
    """As many tiles of 256 rows as fill the card, most with room left in them; then
    a token that only later ones see is NaN, or infinite in one value."""
    rng = np.random.default_rng(32)
    seqs = [(300, 300), (700, 513), (5, 2), (0, 0), (257, 257)]
    c = _case(rng, dtype, seqs, 48, dl, dr, 16, dn, dv)
    clean = _run(c)
    _check(c, seqs, *clean)
    page, sees = int(c["table"].col[(300 + 15) // 16 + 500 // 16]), slice(300 + 500 - 187, 300 + 513)
    some = sum(m for _, m in seqs)
    row = c["cache"][page, 500 % 16].clone()
    for where, value in ((slice(None), float("nan")), (slice(5, 6), -float("inf"))):
        c["cache"][page, 500 % 16] = row
        c["cache"][page, 500 % 16, where] = value
        got = _run(c)
        for a, b in zip(got, clean):
            assert torch.equal(a[:sees.start], b[:sees.start]) and torch.equal(a[sees.stop:some], b[sees.stop:some])
        assert not torch.isfinite(got[0][sees].float()).all(-1).any()


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("count", [256, 257, 700])
def test_many_sequences(count, form):
    """Short texts and empty ones among a few long ones, as many as are cut evenly
    and more; one breaks its batch's rules."""
    rng = np.random.default_rng(count)
    seqs = [(int(n), int(min(n, rng.integers(0, 3)))) for n in rng.integers(0, 90, count)]
    seqs[3], seqs[100], seqs[count - 2] = (900, 2), (0, 0), (1500, 1)
    extra = dict(dn=32, dv=16) if form == "expanded" else {}
    c = _case(rng, BF16, seqs, 2, 64, 8, 16, pad=1, **extra)
    _check(c, seqs, *_run(c))
    c["lengths"][3] = 10 ** 6
    out, lse = _run(c)
    _check(c, seqs, out, lse, skip=(3,))
    start = c["q_rowptr"][3]
    assert torch.isnan(out[start:start + 2]).all() and torch.isnan(lse[start:start + 2]).all()


def test_an_infinite_value_reaches_its_column_alone():
    """The weights do not depend on it where the queries have 0 there: its column is
    infinite in the rows that see it, the other columns are as the formula has them."""
    rng = np.random.default_rng(41)
    seqs = [(100, 30)]
    for dtype in (BF16, F16):
        c = _case(rng, dtype, seqs, 2, 256, 32, 16, pad=0)
        c["q"][:, :, 7] = 0
        page = int(c["table"].col[85 // 16])
        out, lse = _run(c)
        big = 1e30 if dtype == BF16 else 6e4
        c["cache"][page, 85 % 16, 7] = big
        finite = _run(c)
        c["cache"][page, 85 % 16, 7] = float("inf")
        got = _run(c)
        # 0 * inf is NaN in the scores of the rows that see it
        assert torch.isnan(got[1][15:]).all() and torch.equal(got[1][:15], lse[:15])
        assert torch.equal(finite[1], lse) and torch.equal(got[0][:15], out[:15])
        rest = [i for i in range(256) if i != 7]
        assert torch.equal(finite[0][:, :, rest], out[:, :, rest])


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("new", [1, 20])
def test_infinite_and_nan_queries_stay_in_their_rows(new, dtype, form):
    rng = np.random.default_rng(42)
    seqs = [(900, new), (70, new)]
    c = _case(rng, dtype, seqs, 16, 256, 32, 16, pad=0, **(dict(dn=64, dv=64) if form == "expanded" else {}))
    clean = _run(c)
    wild = torch.zeros(2 * new, 16, dtype=torch.bool, device="cuda")
    for t, h, d, x in ((0, 3, 5, float("nan")), (new - 1, 0, 64, float("inf")), (new, 15, 0, -float("inf"))):
        c["q"][t, h, d] = x
        wild[t, h] = True
    for a, b in zip(_run(c), clean):
        assert torch.equal(a[~wild], b[~wild])
        assert not torch.isfinite(a[wild].float().reshape(int(wild.sum()), -1)).all(-1).any()


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_scales_of_the_scores(scale, dtype, form):
    rng = np.random.default_rng(7)
    seqs = [(150, 1), (70, 20)]
    c = _case(rng, dtype, seqs, 2, 128, 32, 16, **(dict(dn=64, dv=64) if form == "expanded" else {}))
    out, lse = _run(c, scale=scale)
    _check(c, seqs, out, lse, scale=scale)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("size", [1e3, 1e5])
@pytest.mark.parametrize("new", [1, 30])
def test_large_scores(new, size, form):
    rng = np.random.default_rng(8)
    seqs = [(190, new)]
    c = _case(rng, BF16, seqs, 1, 128, 32, 16, size=size, **(dict(dn=64, dv=64) if form == "expanded" else {}))
    out, lse = _run(c)
    assert torch.isfinite(out[:new].float()).all() and torch.isfinite(lse[:new]).all()
    _check(c, seqs, out, lse)


def test_ascending_scores():
    """Every tile's scores pass the last one's by more than the reference allows."""
    for form in ("absorbed", "expanded"):
        for dtype in (BF16, F16):
            rng = np.random.default_rng(9)
            seqs = [(400, 2)]
            c = _case(rng, dtype, seqs, 2, 128, 32, 16, **(dict(dn=64, dv=64) if form == "expanded" else {}))
            # a last value that grows with the place, times 1 in the queries
            place = torch.arange(400)
            for s in range(400):
                page = int(c["table"].col[s // 16])
                c["cache"][page, s % 16, -1] = float(place[s]) * 0.25
                c["kept"][0][s, -1] = float(c["cache"][page, s % 16, -1])
            c["q"][:, :, -1] = 16.0
            _check(c, seqs, *_run(c, scale=1.0), scale=1.0)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_bad_batches_give_nan(form):
    rng = np.random.default_rng(36)
    seqs = [(40, 2), (70, 3), (33, 1), (20, 2)]
    c = _case(rng, BF16, seqs, 4, 128, 32, 16, **(dict(dn=64, dv=64) if form == "expanded" else {}))
    shape = (*c["q"].shape[:2], 64 if form == "expanded" else 128)

    def expect(bad, **changed):
        out, lse = _run({**c, **changed}, out=torch.zeros(shape, dtype=BF16, device="cuda"))
        _check(c, seqs, out, lse, skip=(bad,))
        at = sum(m for _, m in seqs[:bad])
        assert torch.isnan(out[at:at + seqs[bad][1]]).all()
        assert torch.isnan(lse[at:at + seqs[bad][1]]).all()
        assert not out[-3:].any()

    t = c["table"]
    for value in (-1, t.ncols, 2 ** 31 - 1, -2 ** 31):
        col = t.col.clone()
        col[int(t.rowptr[1])] = value
        expect(1, table=binding.DeviceCSR(t.nrows, t.ncols, t.rowptr, col, None))
    for length in (2, -1, 81, 10 ** 12):
        lengths = c["lengths"].clone()
        lengths[1] = length
        expect(1, lengths=lengths)
    expect(1, max_len=69)
    rowptr = t.rowptr.clone()
    rowptr[-1] = 10 ** 9
    expect(3, table=binding.DeviceCSR(t.nrows, t.ncols, rowptr, t.col, None))


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_without_work(form):
    rng = np.random.default_rng(38)
    c = _case(rng, BF16, [(5, 1)], 2, 64, 32, 16, pad=0, **(dict(dn=32, dv=32) if form == "expanded" else {}))
    out = torch.full((1, 2, 32 if form == "expanded" else 64), 3.0, dtype=BF16, device="cuda")
    _run(dict(c, q_rowptr=torch.tensor([0, 0]).cuda()), out=out)
    _run(dict(c, max_q=0), out=out)
    none = binding.DeviceCSR(0, c["table"].ncols, torch.zeros(1, dtype=torch.int64).cuda(),
                             torch.zeros(0, dtype=torch.int32).cuda(), None)
    _run(dict(c, table=none, q_rowptr=torch.zeros(1, dtype=torch.int64).cuda(),
              lengths=torch.zeros(0, dtype=torch.int64).cuda()), out=out)
    assert (out == 3.0).all()
    _run(dict(c, q=c["q"][:0], q_rowptr=torch.tensor([0, 0]).cuda()))


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_strides_and_same_bits(form):
    """Head-major queries and results, weights as slices of one tensor; every call alike."""
    rng = np.random.default_rng(12)
    seqs = [(700, 3), (64, 40)]
    c = _case(rng, BF16, seqs, 4, 128, 32, 16, pad=0, **(dict(dn=64, dv=32) if form == "expanded" else {}))
    first = _run(c)
    for _ in range(2):
        again = _run(c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    other = dict(c, q=c["q"].transpose(0, 1).contiguous().transpose(0, 1))
    if form == "expanded":
        both = torch.cat(c["w"], 1)
        other["w"] = [both[:, :64], both[:, 64:]]
    width = first[0].shape[2]
    out = torch.zeros(4, len(c["q"]), width + 8, dtype=BF16, device="cuda").transpose(0, 1)[:, :, :width]
    got = _run(other, out=out)
    assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])


def test_forms_agree():
    """Used together: one model's text, its prompt by the expanded form and its next
    tokens by the absorbed one, each against the other."""
    rng = np.random.default_rng(14)
    heads, dl, dr, dn, dv, page, n = 4, 256, 32, 64, 64, 16, 90
    c = _case(rng, BF16, [(n, n)], heads, dl, dr, page, dn, dv, pad=0)
    out, lse = _run(c)
    _check(c, [(n, n)], out, lse)
    wk, wv = (w.float() for w in c["w"])
    at = 0
    for step in (1, 40, 1, 1, 47):
        new = slice(at, at + step)
        q = c["q"][new].float()
        # the weights multiplied into the queries and the results
        made = torch.cat((torch.bmm(q[:, :, :dn].transpose(0, 1).contiguous(), wk).transpose(0, 1), q[:, :, dn:]), 2)
        sub = dict(c, q=made.to(BF16).contiguous(), max_q=step, max_len=at + step,
                   q_rowptr=torch.tensor([0, step]).cuda(), lengths=torch.tensor([at + step]).cuda())
        del sub["w"]
        o, l = _run(sub)
        o = torch.bmm(o.float().transpose(0, 1).contiguous(), wv.transpose(1, 2).contiguous()).transpose(0, 1)
        # the rounding of the made queries, 2^-8 of their scores of about 1, is the larger part
        assert (o - out[new].float()).abs().max() < 0.06 and (l - lse[new]).abs().max() < 0.03
        at += step
    assert at == n


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_a_captured_step_follows_its_batch(form):
    """Replayed as the texts grow between eager calls, twice at once."""
    rng = np.random.default_rng(13)
    seqs = [(400, 1), (37, 1), (64, 1)]
    c = _case(rng, BF16, seqs, 4, 128, 32, 16, pad=1, **(dict(dn=64, dv=64) if form == "expanded" else {}))
    lengths = c["lengths"].clone()
    c["lengths"] = torch.tensor([3, 2, 1]).cuda()
    _run(c)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, *_run(c)))
    for i in range(4):
        c["lengths"].copy_(lengths * (i + 1) // 4)
        c["q"].copy_(torch.from_numpy(rng.standard_normal(c["q"].shape)).to(BF16))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for (graph, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        o, l = _run(c)
        torch.cuda.synchronize()
        for _, out, lse in graphs:
            assert torch.equal(out[:3], o[:3]) and torch.equal(lse[:3], l[:3]), i
    s = torch.cuda.Stream()
    out, lse = _run(c, stream=s)
    s.synchronize()
    assert torch.equal(out[:3], o[:3]) and torch.equal(lse[:3], l[:3])


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_offsets_past_32_bits(form):
    """Pages 3 GB apart."""
    rng = np.random.default_rng(11)
    c = _case(rng, BF16, [(60, 2)], 2, 64, 32, 16, pad=0, **(dict(dn=32, dv=32) if form == "expanded" else {}))
    t, far = c["cache"], 3 << 29
    big = torch.empty((t.shape[0] - 1) * far + (1 << 16), dtype=BF16, device="cuda")
    view = torch.as_strided(big, t.shape, (far, *t.stride()[1:]))
    view.copy_(t)
    a, b = _run(c), _run(dict(c, cache=view))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals():
    rng = np.random.default_rng(15)
    c = _case(rng, BF16, [(40, 2)], 4, 64, 32, 16, pad=0)
    e = _case(rng, BF16, [(40, 2)], 4, 64, 32, 16, 32, 32, pad=0)
    t = c["table"]
    for x in (c, e):
        for bad in (dict(table=binding.DeviceCSR(1, t.ncols + 1, t.rowptr, t.col, None)),
                    dict(q_rowptr=c["q_rowptr"].int()), dict(lengths=c["lengths"].cpu())):
            with pytest.raises(ValueError):
                _run(dict(x, **bad))
        with pytest.raises(ValueError):
            _run(x, out=torch.empty(2, 4, 8, dtype=BF16, device="cuda"))
        with pytest.raises(ValueError):
            _run(x, lse=torch.empty(2, 3, device="cuda"))
        with pytest.raises(binding.SpgemmError):  # rows that are not 16-byte aligned
            _run(dict(x, q=torch.zeros(2, 4, x["q"].shape[2] + 1, dtype=BF16, device="cuda")[:, :, 1:]))
        width = 64 if x is c else 32
        with pytest.raises(binding.SpgemmError):  # rows of an output that overlap
            _run(x, out=torch.zeros(1, 4, width, dtype=BF16, device="cuda").expand(2, 4, width))
    with pytest.raises(binding.SpgemmError):  # 80 values: not a multiple of 32
        _api().latent_attention(c["q"], c["cache"], t, c["q_rowptr"], c["lengths"], 2, 40, value_dim=80, scale=0.1)
