"""Quantised paged caches on the GPU, through the public calls: what is
written bit by bit, what is read, and attention against the definition in 64
bits with a bound per element."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from spgemm_irregular_matrices_amd import binding  # noqa: E402
from tests import attention_ref as ref  # noqa: E402
from tests import cache_ref as cref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FORMS = ["e4m3", "e2m1"]
SEQS = [(1, 1), (33, 1), (40, 7), (5, 5), (0, 0), (130, 2), (200, 33), (64, 64)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from spgemm_irregular_matrices_amd import cache
    cache.load()


def _cache(*args, **more):
    from spgemm_irregular_matrices_amd import cache
    return cache.QuantizedCache(*args, **more)


def _index(rng, seqs, page, pad):
    """Tables of a batch: (cached tokens, new ones among them) per sequence."""
    count = [(n + page - 1) // page for n, _ in seqs]
    pool = sum(count) + 2
    order = rng.permutation(pool)[:sum(count)]
    rowptr = np.concatenate([[0], np.cumsum(count)]).astype(np.int64)
    start = np.concatenate([[0], np.cumsum([m for _, m in seqs])]).astype(np.int64)
    table = binding.DeviceCSR(len(seqs), pool, torch.from_numpy(rowptr).cuda(),
                              torch.from_numpy(order.astype(np.int32)).cuda(), None)
    return dict(pages=table, q_rowptr=torch.from_numpy(start).cuda(),
                lengths=torch.tensor([n for n, _ in seqs], dtype=torch.int64).cuda(),
                max_q=max(m for _, m in seqs), max_len=max(n for n, _ in seqs)), pool, order, rowptr, \
        int(start[-1]) + pad


def _bytes(shape, layout):
    """A byte tensor of that shape in one of several layouts, full of 0xa5."""
    pages, slots, heads, width = shape
    if layout == "heads":
        return torch.full((pages, heads, slots, width), 0xa5, dtype=torch.uint8, device="cuda").transpose(1, 2)
    if layout == "gaps":
        whole = torch.full((pages, slots, heads + 1, width + 16), 0xa5, dtype=torch.uint8, device="cuda")
        return whole[:, :, :heads, :width]
    return torch.full(shape, 0xa5, dtype=torch.uint8, device="cuda")


def _empty(pool, page, heads, d, form, layout="slots"):
    wide = d if form == "e4m3" else d // 2
    return _cache(*(_bytes((pool, page, heads, w), layout) for w in (wide, d // 32) * 2), form)


def _filled(rng, seqs, d, hkv, page, form, pad=3, layout="slots", spread=0.0):
    """A cache with random codes and scales in every sequence's places, NaN in all
    others, and the values of every sequence."""
    index, pool, order, rowptr, tokens = _index(rng, seqs, page, pad)
    c = _empty(pool, page, hkv, d, form, layout)
    kept = []
    for codes, scales in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)):
        cc = np.full(codes.shape, 0x7f if form == "e4m3" else 0x55, dtype=np.uint8)
        ss = np.full(scales.shape, 255, dtype=np.uint8)
        mine = []
        for s, (n, _) in enumerate(seqs):
            x = rng.standard_normal((n, hkv, d)) * np.exp(spread * rng.standard_normal((n, hkv, 1)))
            a, b = cref.quantize(x, form)
            at = np.arange(n)
            where = order[rowptr[s] + at // page], at % page
            cc[where], ss[where] = cref.pack(a.astype(np.int64), form), b
            mine.append(cref.values(a.astype(np.int64), b, form))
        codes.copy_(torch.from_numpy(cc))
        scales.copy_(torch.from_numpy(ss))
        kept.append(mine)
    return c, index, kept, tokens


# ---------------------------------------------------------------- writing, reading
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,d,heads,page,layout", [
    (BF16, 128, 2, 16, "slots"), (F16, 32, 3, 1, "heads"), (F32, 64, 1, 7, "gaps"), (BF16, 96, 5, 24, "heads"),
    (F32, 256, 2, 64, "slots"), (F16, 192, 1, 5, "gaps"), (F32, 160, 9, 3, "slots")])
def test_written_codes_are_the_nearest(dtype, d, heads, page, layout, form):
    rng = np.random.default_rng(d + page)
    index, pool, order, rowptr, tokens = _index(rng, SEQS, page, 3)
    # magnitudes from the type's smallest to its largest, ties, zeros and wild blocks
    wide = {BF16: 80, F32: 80, F16: 9}[dtype]
    x = rng.standard_normal((2, tokens, heads, d)) * np.exp2(rng.uniform(-wide, wide, (2, tokens, heads, 1)))
    grid = rng.integers(-60, 61, x.shape) * 0.125 * np.exp2(rng.integers(-9, 9, (2, tokens, heads, 1)).astype(float))
    x = np.where(rng.random((2, tokens, heads, 1)) < 0.5, grid, x)
    x[:, :, :, ::7] *= 2.0 ** -12
    x[:, 0] = 0.0
    x[0, 2, 0, 3], x[1, 3, 0, d - 1], x[1, 4, 0, 0] = np.nan, np.inf, -np.inf
    x[0, 6, 0] = 1e-38 if dtype != F16 else 2.0 ** -24
    x[1, 7, 0, :32] = {BF16: 3.3e38, F32: 3.4e38, F16: 65504.0}[dtype]
    kv = torch.from_numpy(x).to(dtype).cuda()
    fused = torch.cat((kv[0], kv[1]), 1)  # as one projection leaves them
    c = _empty(pool, page, heads, d, form, layout)
    c.write(fused[:, :heads], fused[:, heads:], **index)
    for codes, scales, part in ((c.k_codes, c.k_scales, kv[0]), (c.v_codes, c.v_scales, kv[1])):
        want_c, want_s = np.full(codes.shape, 0xa5, np.uint8), np.full(scales.shape, 0xa5, np.uint8)
        at = 0
        for s, (n, m) in enumerate(SEQS):
            a, b = cref.quantize(ref.f64(part[at:at + m]), form)
            where = order[rowptr[s] + np.arange(n - m, n) // page], np.arange(n - m, n) % page
            a = np.where(np.repeat(b == 255, 32, -1), 0, a).astype(np.int64)
            want_c[where], want_s[where] = cref.pack(a, form), b
            at += m
        assert np.array_equal(scales.cpu().numpy(), want_s)
        assert np.array_equal(codes.cpu().numpy(), want_c)
    # and back, into rows of other strides; rows behind the last sequence stay
    out = torch.full((tokens, 2 * heads, d), 7.0, dtype=dtype, device="cuda")
    k, v = c.read(**index, k=out[:, heads:], v=out[:, :heads])
    for got, part in ((k, kv[0]), (v, kv[1])):
        a, b = cref.quantize(ref.f64(part[:tokens - 3]), form)
        want = torch.from_numpy(cref.values(a.astype(np.int64), b, form)).to(dtype)
        assert torch.equal(got[:-3].cpu().nan_to_num(nan=5.0), want.nan_to_num(nan=5.0))
        assert (got[-3:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("form", FORMS)
def test_every_code_and_scale_is_read(form, dtype):
    """All codes with all scales: a cache may come from elsewhere."""
    n = 256
    d = 256 if form == "e4m3" else 32
    codes = np.tile(np.arange(d) if form == "e4m3" else np.arange(32) % 16, (n, 1, 1))
    scales = np.tile(np.arange(n)[:, None, None], (1, 1, d // 32))
    put = lambda x: torch.from_numpy(np.ascontiguousarray(x).astype(np.uint8)).cuda()[None]  # noqa: E731
    c = _cache(put(cref.pack(codes, form)), put(scales), put(cref.pack(codes[::-1], form)), put(scales), form)
    table = binding.DeviceCSR(1, 1, torch.tensor([0, 1]).cuda(), torch.zeros(1, dtype=torch.int32).cuda(), None)
    k, v = c.read(table, torch.tensor([0, n]).cuda(), torch.tensor([n]).cuda(), n, n, tokens=n, dtype=dtype)
    want = torch.from_numpy(cref.values(codes, scales, form)).to(dtype)
    assert torch.equal(k.cpu().nan_to_num(nan=5.0, posinf=1e4, neginf=-1e4),
                       want.nan_to_num(nan=5.0, posinf=1e4, neginf=-1e4))
    assert torch.equal(k.isnan(), v.isnan())


def test_reading_whole_texts_and_defaults():
    rng = np.random.default_rng(2)
    seqs = [(90, 90), (1, 1), (33, 33)]
    c, index, (ks, vs), tokens = _filled(rng, seqs, 64, 2, 16, "e4m3", pad=0)
    k, v = c.read(**index, tokens=tokens)
    assert k.dtype == BF16 and k.shape == (124, 2, 64)
    assert np.array_equal(ref.f64(k), np.concatenate(ks)) and np.array_equal(ref.f64(v), np.concatenate(vs))
    k32, _ = c.read(**index, tokens=tokens, dtype=F32)
    assert torch.equal(k32, k.float())
    with pytest.raises(ValueError, match="tokens"):
        c.read(**index)


def test_many_sequences_and_empty_ones():
    """The search for a token's sequence: thousands of them, most without new tokens."""
    rng = np.random.default_rng(3)
    m = np.where(rng.random(5000) < 0.9, 0, rng.integers(1, 4, 5000))
    seqs = [(int(x), int(x)) for x in m]
    index, pool, order, rowptr, tokens = _index(rng, seqs, 4, 2)
    x = torch.randn(tokens, 1, 32, device="cuda", dtype=BF16)
    c = _empty(pool, 4, 1, 32, "e4m3")
    c.write(x, x, **index)
    k, v = c.read(**index, tokens=tokens)
    codes, scales = cref.quantize(ref.f64(x), "e4m3")
    want = cref.values(codes.astype(np.int64), scales, "e4m3")
    assert np.array_equal(ref.f64(k)[:-2], want[:-2]) and np.array_equal(ref.f64(v)[:-2], want[:-2])


def test_bad_batches_write_nothing_and_read_nan():
    rng = np.random.default_rng(4)
    seqs = [(40, 2), (70, 3), (33, 1), (20, 2)]
    index, pool, order, rowptr, tokens = _index(rng, seqs, 16, 3)
    x = torch.randn(tokens, 2, 64, device="cuda", dtype=BF16)
    starts = np.concatenate([[0], np.cumsum([m for _, m in seqs])])
    t = index["pages"]

    def expect(bad, tokens_bad=None, **changed):
        c, good = _empty(pool, 16, 2, 64, "e4m3"), _empty(pool, 16, 2, 64, "e4m3")
        good.write(x, x, **index)
        k0, v0 = good.read(**index, k=torch.zeros_like(x), v=torch.zeros_like(x))
        c.write(x, x, **{**index, **changed})
        rows = np.arange(starts[bad], starts[bad + 1]) if tokens_bad is None else starts[bad] + np.array(tokens_bad, dtype=np.int64)
        n, m = seqs[bad]
        places = n - m + rows - starts[bad]
        where = torch.from_numpy(order[rowptr[bad] + places // 16]).cuda(), torch.from_numpy(places % 16).cuda()
        for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
            want = getattr(good, name).clone()
            want[where] = 0xa5
            assert torch.equal(getattr(c, name), want), name
        k, v = good.read(**{**index, **changed}, k=torch.zeros_like(x), v=torch.zeros_like(x))
        k0[rows], v0[rows] = float("nan"), float("nan")
        assert torch.equal(k.nan_to_num(nan=99.0), k0.nan_to_num(nan=99.0))
        assert torch.equal(v.nan_to_num(nan=99.0), v0.nan_to_num(nan=99.0))

    for value in (-1, t.ncols, 2 ** 31 - 1, -2 ** 31):
        col = t.col.clone()
        col[int(rowptr[1]) + 4] = value  # the page of tokens 64 to 69, the new ones
        expect(1, pages=binding.DeviceCSR(t.nrows, t.ncols, t.rowptr, col, None))
        col = t.col.clone()
        col[int(rowptr[1])] = value  # a page that no new token is in
        expect(1, [], pages=binding.DeviceCSR(t.nrows, t.ncols, t.rowptr, col, None))
    for length in (2, -1, 81, 10 ** 12):
        lengths = index["lengths"].clone()
        lengths[1] = length
        expect(1, lengths=lengths)
    expect(1, max_len=69)
    table = t.rowptr.clone()
    table[-1] = 10 ** 9
    expect(3, pages=binding.DeviceCSR(t.nrows, t.ncols, table, t.col, None))


def test_without_work():
    rng = np.random.default_rng(5)
    index, pool, order, rowptr, tokens = _index(rng, [(5, 1)], 16, 0)
    c = _empty(pool, 16, 1, 64, "e4m3")
    x = torch.ones(tokens, 1, 64, device="cuda", dtype=BF16)
    out, q = torch.full_like(x, 3.0), torch.ones(tokens, 2, 64, device="cuda", dtype=BF16)
    none = dict(pages=binding.DeviceCSR(0, pool, torch.zeros(1, dtype=torch.int64).cuda(),
                                        torch.zeros(0, dtype=torch.int32).cuda(), None),
                q_rowptr=torch.zeros(1, dtype=torch.int64).cuda(), lengths=torch.zeros(0, dtype=torch.int64).cuda())
    for changed in (dict(q_rowptr=torch.tensor([0, 0]).cuda()), dict(max_q=0), none):
        batch = {**index, **changed}
        c.write(x, x, **batch)
        c.read(**batch, k=out, v=out.clone())
        got, _ = c.attention(q, **batch, out=torch.full_like(q, 3.0))
        assert (got == 3.0).all()
    assert (out == 3.0).all() and (c.k_codes == 0xa5).all() and (c.v_scales == 0xa5).all()
    c.write(x[:0], x[:0], **{**index, "q_rowptr": torch.tensor([0, 0]).cuda()})


# ---------------------------------------------------------------- attention
def _check(c, index, kept, seqs, q, out, lse, scale, skip=()):
    dtype = q.dtype
    parts = cref.PARTS[dtype]
    at = 0
    for s, (n, m) in enumerate(seqs):
        if m and s not in skip:
            o, l, oe, le = cref.attend(ref.f64(q[at:at + m]), kept[0][s], kept[1][s], n - m, scale, dtype,
                                       parts * q.shape[2], cref.WEIGHT[dtype], parts)
            ref.check(out[at:at + m], o, oe, f"out of sequence {s}")
            ref.check(lse[at:at + m], l, le, f"lse of sequence {s}")
        at += m


def _query(rng, tokens, hq, d, dtype, scale=1.0):
    return torch.from_numpy(scale * rng.standard_normal((tokens, hq, d))).to(dtype).cuda()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,d,hq,hkv,page,layout", [
    (BF16, 64, 4, 2, 16, "slots"), (BF16, 128, 8, 1, 1, "heads"), (F16, 64, 7, 1, 24, "gaps"),
    (F32, 64, 3, 3, 7, "slots"), (BF16, 32, 2, 2, 64, "slots"), (F16, 256, 16, 1, 32, "slots"),
    (F32, 192, 4, 2, 128, "gaps"), (BF16, 96, 20, 1, 5, "heads"), (F32, 128, 2, 1, 16, "slots"),
    (BF16, 224, 2, 1, 9, "slots"), (F16, 160, 5, 1, 11, "slots"), (F32, 32, 1, 1, 3, "slots")])
def test_attention(dtype, d, hq, hkv, page, layout, form):
    rng = np.random.default_rng(hq * 1000 + page)
    c, index, kept, tokens = _filled(rng, SEQS, d, hkv, page, form, layout=layout, spread=0.5)
    q = _query(rng, tokens, hq, d, dtype)
    lse = torch.full((tokens, hq), 9.0, device="cuda")
    out, lse = c.attention(q, **index, out=torch.full_like(q, 7.0), lse=lse, scale=d ** -0.5)
    _check(c, index, kept, SEQS, q, out, lse, d ** -0.5)
    assert (out[-3:] == 7.0).all() and (lse[-3:] == 9.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 1), (128, 2, 2), (128, 20, 1), (256, 4, 1)])
def test_single_tokens(d, hq, hkv, dtype, form):
    """The next token of sequences of one to 700 cached ones, pieces joined."""
    rng = np.random.default_rng(31)
    seqs = [(n, 1) for n in (1, 2, 31, 32, 33, 63, 64, 65, 500, 700)]
    c, index, kept, tokens = _filled(rng, seqs, d, hkv, 16, form)
    q = _query(rng, tokens, hq, d, dtype)
    out, lse = c.attention(q, **index)
    _check(c, index, kept, seqs, q, out, lse, d ** -0.5)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("new", [8, 24, 120])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("d", [64, 128, 192])
def test_chunk_sizes(d, dtype, new, form):
    """Chunks of 16 to 240 rows to a key head, in the tiles of single wavefronts
    and of work groups; then a wild key and value that only later tokens see."""
    rng = np.random.default_rng(d + new)
    seqs = [(40 + new, new), (new, new), (310, max(1, new // 3)), (3, 1)]
    c, index, kept, tokens = _filled(rng, seqs, d, 2, 16, form)
    q = _query(rng, tokens, 4, d, dtype)
    clean = c.attention(q, **index)
    _check(c, index, kept, seqs, q, *clean, d ** -0.5)
    at = 40 + new // 2  # seen by the first sequence's tokens from new // 2 on
    page = int(index["pages"].col[at // 16])
    c.k_scales[page, at % 16], c.v_scales[page, at % 16] = 255, 255
    got = c.attention(q, **index)
    sees = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    sees[new // 2:new] = True
    some = sum(m for _, m in seqs)
    for a, b in zip(got, clean):
        assert torch.equal(a[:some][~sees[:some]], b[:some][~sees[:some]])
    assert not torch.isfinite(got[0][sees].float()).any()
    assert not torch.isfinite(got[1][sees]).any()


def test_long_texts_in_pieces():
    rng = np.random.default_rng(6)
    seqs = [(3000, 40), (2500, 1), (64, 2), (1111, 30)]
    for dtype, form in ((BF16, "e4m3"), (F16, "e2m1")):
        c, index, kept, tokens = _filled(rng, seqs, 64, 1, 16, form)
        q = _query(rng, tokens, 2, 64, dtype)
        out, lse = c.attention(q, **index)
        _check(c, index, kept, seqs, q, out, lse, 0.125)


@pytest.mark.parametrize("count", [256, 257, 600])
def test_attention_over_many_sequences(count):
    """Short texts and empty ones among a few long ones, as many as are cut evenly
    and more; one breaks its batch's rules."""
    rng = np.random.default_rng(count)
    seqs = [(int(n), int(min(n, rng.integers(0, 3)))) for n in rng.integers(0, 90, count)]
    seqs[3], seqs[100], seqs[count - 2] = (900, 2), (0, 0), (1500, 1)
    c, index, kept, tokens = _filled(rng, seqs, 64, 2, 16, "e4m3", pad=1)
    q = _query(rng, tokens, 6, 64, BF16)
    _check(c, index, kept, seqs, q, *c.attention(q, **index), 64 ** -0.5)
    lengths = index["lengths"].clone()
    lengths[3] = 10 ** 6
    out, lse = c.attention(q, **{**index, "lengths": lengths})
    _check(c, index, kept, seqs, q, out, lse, 64 ** -0.5, skip=(3,))
    start = index["q_rowptr"][3]
    assert torch.isnan(out[start:start + 2]).all() and torch.isnan(lse[start:start + 2]).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
def test_wild_tokens_of_evenly_cut_texts(dtype, form):
    """A block of a long text's token becomes NaN: so do its values in the rows that
    see it, whichever range it lies in, and no other row changes."""
    rng = np.random.default_rng(33)
    seqs = [(2100, 4), (60, 3), (1000, 4)]
    c, index, kept, tokens = _filled(rng, seqs, 128, 1, 16, form, pad=0)
    q = _query(rng, tokens, 4, 128, dtype)
    clean = c.attention(q, **index)
    _check(c, index, kept, seqs, q, *clean, 128 ** -0.5)
    for at in (0, 1030, 2098):
        page = int(index["pages"].col[at // 16])
        old = c.v_scales[page, at % 16].clone()
        c.v_scales[page, at % 16, 0, 2] = 255
        out, lse = c.attention(q, **index)
        first = max(0, at - 2096)
        assert torch.isnan(out[first:4, :, 64:96]).all() and torch.equal(lse, clean[1])
        out[first:4, :, 64:96] = clean[0][first:4, :, 64:96]
        assert torch.equal(out[:first], clean[0][:first]) and torch.equal(out[4:], clean[0][4:])
        # its other values are added apart from the matrix products, by one product and
        # one sum in floats each: 2 roundings of the 2 * count that the bound has
        _check(c, index, kept, seqs, q, out, lse, 128 ** -0.5)
        c.v_scales[page, at % 16] = old


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
def test_scales_of_the_scores(dtype, scale):
    rng = np.random.default_rng(7)
    seqs = [(50, 1), (70, 20)]
    c, index, kept, tokens = _filled(rng, seqs, 64, 1, 16, "e4m3")
    q = _query(rng, tokens, 2, 64, dtype)
    out, lse = c.attention(q, **index, scale=scale)
    _check(c, index, kept, seqs, q, out, lse, scale)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("size", [1e3, 1e5])
@pytest.mark.parametrize("new", [1, 30])
def test_large_scores(dtype, size, new):
    """Scores whose rounding in floats decides: the largest key's weight is 1."""
    rng = np.random.default_rng(8)
    seqs = [(90, new)]
    c, index, kept, tokens = _filled(rng, seqs, 64, 1, 16, "e4m3")
    q = _query(rng, tokens, 1, 64, dtype, size)
    out, lse = c.attention(q, **index)
    assert torch.isfinite(out[:new].float()).all() and torch.isfinite(lse[:new]).all()
    _check(c, index, kept, seqs, q, out, lse, 0.125)


def test_infinite_and_nan_queries_stay_in_their_rows():
    rng = np.random.default_rng(9)
    for dtype in (BF16, F16, F32):
        for new in (2, 40):
            seqs = [(60, new), (50, new)]
            c, index, kept, tokens = _filled(rng, seqs, 64, 1, 16, "e4m3")
            q = _query(rng, tokens, 2, 64, dtype)
            clean = c.attention(q, **index)
            q[0, 1, 5], q[1, 0, 63] = float("nan"), float("inf")
            out, lse = c.attention(q, **index)
            hit = torch.zeros(tokens, 2, dtype=torch.bool, device="cuda")
            hit[0, 1] = hit[1, 0] = True
            n = 2 * new
            assert torch.equal(out[:n][~hit[:n]], clean[0][:n][~hit[:n]])
            assert torch.equal(lse[:n][~hit[:n]], clean[1][:n][~hit[:n]])
            assert torch.isnan(out[0, 1]).all() and not torch.isfinite(lse[1, 0])


def test_bad_batches_give_nan():
    rng = np.random.default_rng(36)
    seqs = [(40, 2), (70, 3), (33, 1), (20, 2)]
    for hq in (2, 32):  # both kernels
        c, index, kept, tokens = _filled(rng, seqs, 64, 1, 16, "e4m3")
        q = _query(rng, tokens, hq, 64, BF16)
        t = index["pages"]

        def expect(bad, **changed):
            out, lse = c.attention(q, **{**index, **changed}, out=torch.zeros_like(q))
            _check(c, index, kept, seqs, q, out, lse, 0.125, skip=(bad,))
            at = sum(m for _, m in seqs[:bad])
            assert torch.isnan(out[at:at + seqs[bad][1]]).all()
            assert torch.isnan(lse[at:at + seqs[bad][1]]).all()
            assert not out[-3:].any()

        for value in (-1, t.ncols, 2 ** 31 - 1, -2 ** 31):
            col = t.col.clone()
            col[int(t.rowptr[1])] = value
            expect(1, pages=binding.DeviceCSR(t.nrows, t.ncols, t.rowptr, col, None))
        for length in (2, -1, 81, 10 ** 12):
            lengths = index["lengths"].clone()
            lengths[1] = length
            expect(1, lengths=lengths)
        expect(1, max_len=69)
        rowptr = t.rowptr.clone()
        rowptr[-1] = 10 ** 9
        expect(3, pages=binding.DeviceCSR(t.nrows, t.ncols, rowptr, t.col, None))


def test_same_bits_every_time():
    rng = np.random.default_rng(10)
    seqs = [(900, 3), (700, 1), (64, 40)]
    c, index, kept, tokens = _filled(rng, seqs, 128, 2, 16, "e4m3", pad=0)
    q = _query(rng, tokens, 8, 128, BF16)
    first = c.attention(q, **index)
    for _ in range(3):
        again = c.attention(q, **index)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_offsets_past_32_bits():
    """Pages 1.5 GB apart: places in bytes need 33 bits."""
    rng = np.random.default_rng(11)
    seqs = [(60, 2)]
    c, index, kept, tokens = _filled(rng, seqs, 64, 1, 16, "e4m3", pad=0)
    pool, far = c.npages, 3 << 29
    big = torch.empty((pool - 1) * far + (1 << 16), dtype=torch.uint8, device="cuda")
    parts, at = [], 0
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        view = torch.as_strided(big, t.shape, (far, *t.stride()[1:]), at)
        view.copy_(t)
        parts.append(view)
        at += t[0].numel()
    wide = _cache(*parts, "e4m3")
    q = _query(rng, tokens, 2, 64, BF16)
    for a, b in ((wide.attention(q, **index), c.attention(q, **index)),
                 (wide.read(**index, tokens=tokens), c.read(**index, tokens=tokens))):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = torch.randn(tokens, 1, 64, device="cuda", dtype=BF16)
    c.write(x, -x, **index)
    wide.write(x, -x, **index)
    for a, b in zip(parts, (c.k_codes, c.k_scales, c.v_codes, c.v_scales)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- used together
@pytest.mark.parametrize("form", FORMS)
def test_a_text_grows(form):
    """Chunks are written and attended to as a server does, then read back: the
    attention is that of what is read, by the paged attention of 16-bit caches too."""
    from spgemm_irregular_matrices_amd import attention
    rng = np.random.default_rng(12)
    page, d, hkv, hq = 16, 64, 2, 4
    seqs = [(150, 150), (90, 90)]
    index, pool, order, rowptr, _ = _index(rng, seqs, page, 0)
    c = _empty(pool, page, hkv, d, form)
    done = [0, 0]
    for steps in ((40, 64), (1, 1), (1, 0), (70, 24), (1, 1), (37, 0)):
        done = [a + b for a, b in zip(done, steps)]
        start = torch.tensor([0, steps[0], sum(steps)]).cuda()
        batch = dict(index, q_rowptr=start, lengths=torch.tensor(done).cuda(), max_q=max(steps), max_len=max(done))
        k, v = (_query(rng, sum(steps), hkv, d, BF16) for _ in range(2))
        q = _query(rng, sum(steps), hq, d, BF16)
        c.write(k, v, **batch)
        out, lse = c.attention(q, **batch)
        whole = dict(batch, q_rowptr=torch.tensor([0, done[0], sum(done)]).cuda(), max_q=max(done))
        kk, vv = c.read(**whole, tokens=sum(done))
        ks, vs = ([ref.f64(x[:done[0]]), ref.f64(x[done[0]:])] for x in (kk, vv))
        _check(c, batch, (ks, vs), [(n, m) for n, m in zip(done, steps)], q, out, lse, 0.125)
        plain = torch.zeros(2, pool, page, hkv, d, dtype=BF16, device="cuda")
        for s in range(2):
            at = np.arange(done[s])
            where = torch.from_numpy(order[rowptr[s] + at // page]).cuda(), torch.from_numpy(at % page).cuda()
            plain[0][where], plain[1][where] = (torch.from_numpy(x[s]).to(BF16).cuda() for x in (ks, vs))
        o, l = attention.paged_attention(q, plain[0], plain[1], batch["pages"], start, batch["lengths"],
                                         max(steps), max(done))
        assert (out.float() - o.float()).abs().max() < 0.05 and (lse - l).abs().max() < 1e-4
    # new tokens read back as they were rounded
    codes, scales = cref.quantize(ref.f64(k), form)
    last = c.read(**batch, tokens=len(k))[0]
    assert np.array_equal(ref.f64(last), cref.values(codes.astype(np.int64), scales, form))


def test_a_captured_step_follows_its_batch():
    """Write and attention of a step in one graph, replayed as the texts grow
    between eager calls, and two graphs that run at once."""
    rng = np.random.default_rng(13)
    seqs = [(100, 1), (37, 1), (64, 1)]
    c, index, kept, tokens = _filled(rng, seqs, 64, 2, 16, "e4m3", pad=1)
    lengths = index["lengths"].clone()
    index["lengths"] = torch.tensor([3, 2, 1]).cuda()
    k, v, q = (_query(rng, tokens, h, 64, BF16) for h in (2, 2, 8))

    def step():
        c.write(k, v, **index)
        return c.attention(q, **index)

    step()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, lse = step()
            back = c.read(**index, tokens=tokens)
        graphs.append((graph, out, lse, back))
    for i in range(4):
        index["lengths"].copy_(lengths * (i + 1) // 4)
        for t in (k, v, q):
            t.copy_(_query(rng, *t.shape, BF16))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for (graph, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        o, l = step()
        b = c.read(**index, tokens=tokens)
        torch.cuda.synchronize()
        for _, out, lse, back in graphs:
            assert torch.equal(out[:3], o[:3]) and torch.equal(lse[:3], l[:3]), i
            assert torch.equal(back[0][:3], b[0][:3]) and torch.equal(back[1][:3], b[1][:3]), i


def test_another_stream():
    rng = np.random.default_rng(14)
    seqs = [(500, 3), (90, 3)]
    c, index, kept, tokens = _filled(rng, seqs, 128, 1, 16, "e2m1", pad=0)
    q = _query(rng, tokens, 4, 128, F16)
    want = c.attention(q, **index)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, lse = c.attention(q, **index, stream=s)
    k, v = c.read(**index, tokens=tokens, stream=s)
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    k0, v0 = c.read(**index, tokens=tokens)
    c.write(k, v, **index, stream=s)  # what is read is what would be written again
    s.synchronize()
    assert torch.equal(k, k0) and torch.equal(v, v0)
    a, b = c.read(**index, tokens=tokens)
    assert torch.equal(a, k0) and torch.equal(b, v0)


# ---------------------------------------------------------------- refusals
def test_refusals():
    rng = np.random.default_rng(15)
    seqs = [(40, 2)]
    c, index, kept, tokens = _filled(rng, seqs, 64, 2, 16, "e4m3", pad=0)
    q = _query(rng, tokens, 4, 64, BF16)
    x = _query(rng, tokens, 2, 64, BF16)
    t = index["pages"]
    for bad in (dict(pages=binding.DeviceCSR(1, t.ncols + 1, t.rowptr, t.col, None)),
                dict(q_rowptr=index["q_rowptr"].int()), dict(q_rowptr=index["q_rowptr"].cpu()),
                dict(lengths=index["lengths"][:0])):
        for call in (lambda b: c.attention(q, **b), lambda b: c.write(x, x, **b),
                     lambda b: c.read(**b, tokens=tokens)):
            with pytest.raises(ValueError):
                call({**index, **bad})
    with pytest.raises(binding.SpgemmError):  # three query heads on two key heads
        c.attention(q[:, :3], **index)
    with pytest.raises(ValueError):
        c.attention(q, **index, out=torch.empty_like(q).float())
    with pytest.raises(ValueError):
        c.attention(q, **index, lse=torch.empty(tokens, 3, device="cuda"))
    with pytest.raises(ValueError):
        c.read(**index, k=x, dtype=F16)
    with pytest.raises(binding.SpgemmError):  # rows of an output that overlap
        c.read(**index, k=x[:1].expand(tokens, 2, 64), v=x)
    with pytest.raises(binding.SpgemmError):  # rows that are not 16-byte aligned
        c.write(torch.zeros(tokens, 2, 65, device="cuda", dtype=BF16)[:, :, 1:], x, **index)
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError):
            c.attention(q, **index, stream=torch.cuda.Stream(1))
