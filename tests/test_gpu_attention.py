"""Attention over a CSR mask and over a paged cache on the GPU, through the
public calls, against the definition in 64 bits with a bound per element."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import attention_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from spgemm_irregular_matrices_amd import attention
    attention.load()


def _api():
    from spgemm_irregular_matrices_amd import attention
    return attention


def _rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(dtype).cuda()


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 0, 64, 65, 127, 128, 129, 200, 300, 5, 0]


def _case(rng, dtype, d, hq, hkv, nk=301, lengths=LENGTHS, repeat=False):
    rows = ref.mask(lengths, nk, rng, repeat)
    nq = len(rows)
    q, k, v, dout = (_rand(rng, s, dtype) for s in ((nq, hq, d), (nk, hkv, d), (nk, hkv, d),
                                                    (nq, hq, d)))
    unread = np.setdiff1d(np.arange(nk), np.concatenate(rows).astype(int))
    k[unread] = float("nan")  # rows that no entry names reach nothing
    v[unread] = float("inf")
    return rows, q, k, v, dout


def _check_both(rows, q, k, v, dout, nk, scale, grads=True):
    api = _api()
    dtype = q.dtype
    with api.AttentionPlan(ref.csr(rows, nk), backward=grads) as plan:
        out, lse = plan.forward(q, k, v, scale=scale)
        a = [ref.f64(x) for x in (q, k, v)]
        o, l, oe, le = ref.forward(*a, rows, scale, dtype)
        ref.check(out, o, oe, "out")
        ref.check(lse, l, le, "lse")
        if not grads:
            return
        got = plan.backward(dout, q, k, v, out, lse, scale=scale)
        want, err = ref.backward(*a, ref.f64(out), ref.f64(lse), ref.f64(dout), rows, scale, dtype)
        for name, x, w, e in zip(("dq", "dk", "dv"), got, want, err):
            ref.check(x, w, e, name)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("d", [8, 40, 64, 72, 128, 136, 256])
def test_head_dims(dtype, d):
    rng = np.random.default_rng(d)
    rows, q, k, v, dout = _case(rng, dtype, d, 4, 2)
    _check_both(rows, q, k, v, dout, 301, d ** -0.5)


@pytest.mark.parametrize("dtype,hq,hkv", [(BF16, 1, 1), (BF16, 7, 1), (BF16, 16, 1), (F16, 20, 1),
                                          (F32, 6, 3), (BF16, 34, 2), (F16, 3, 3), (F32, 17, 1)])
def test_head_layouts(dtype, hq, hkv):
    rng = np.random.default_rng(hq * 100 + hkv)
    rows, q, k, v, dout = _case(rng, dtype, 64, hq, hkv)
    _check_both(rows, q, k, v, dout, 301, 0.125)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("hq,hkv,kind", [(1, 1, "short"), (8, 2, "short"), (3, 1, "band"), (16, 2, "band"),
                                         (5, 1, "band"), (18, 2, "band"), (2, 1, "long"), (4, 1, "hub")])
def test_rows_that_share_work(dtype, hq, hkv, kind):
    """Ascending rows, four of which share tiles: short ones, neighbours in a
    band (with wild values in keys that only some of the four see), long ones
    without common columns, and one long row among empty ones."""
    rng = np.random.default_rng(hq * 10 + len(kind))
    nk = 700
    if kind == "short":
        rows = [np.sort(r) for r in ref.mask([0, 3, 0, 40, 17, 1, 1, 2, 0, 0, 0, 0, 33, 32, 31, 5, 6], nk, rng)]
    elif kind == "band":
        rows = [np.arange(max(0, i - 150), i + 1) for i in range(203)]
        nk = 203
    elif kind == "long":
        rows = [np.arange(i % 4, nk, 4) for i in range(9)]
    else:
        rows = [np.arange(nk) if i == 6 else np.zeros(0, int) for i in range(14)]
    nq = len(rows)
    q, k, v, dout = (_rand(rng, s, dtype) for s in ((nq, hq, 64), (nk, hkv, 64), (nk, hkv, 64), (nq, hq, 64)))
    _check_both(rows, q, k, v, dout, nk, 0.125)
    # a NaN key and an infinite value reach the rows that store them and no others
    api = _api()
    bad = 2 if kind != "short" else int(rows[3][7])
    with api.AttentionPlan(ref.csr(rows, nk), backward=True) as plan:
        out, lse = plan.forward(q, k, v)
        clean = (out, lse, *plan.backward(dout, q, k, v, out, lse))
        k[bad], v[bad] = float("nan"), float("inf")
        out, lse = plan.forward(q, k, v)
        got = (out, lse, plan.backward(dout, q, k, v, out, lse)[0])
    has = torch.tensor([bad in set(r.tolist()) for r in rows]).cuda()
    assert has.any() and (kind == "hub" or not has.all())
    for a, b in zip(got, clean):
        assert torch.equal(a[~has], b[~has])
        assert not torch.isfinite(a[has].float()).any() if a.dim() == 2 else \
            not torch.isfinite(a[has].float()).all(2).any()


def test_float_head_dim_of_four():
    rng = np.random.default_rng(4)
    rows, q, k, v, dout = _case(rng, F32, 4, 2, 1)
    _check_both(rows, q, k, v, dout, 301, 0.5)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
def test_repeated_columns_count_as_keys(dtype):
    rng = np.random.default_rng(11)
    rows, q, k, v, dout = _case(rng, dtype, 64, 2, 1, nk=40, repeat=True)
    _check_both(rows, q, k, v, dout, 40, 0.125)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales(scale):
    rng = np.random.default_rng(12)
    rows, q, k, v, dout = _case(rng, BF16, 64, 2, 2)
    _check_both(rows, q, k, v, dout, 301, scale)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
def test_long_rows_and_columns(dtype):
    """Rows and columns of many pieces: one row sees everything, one column is seen by all."""
    rng = np.random.default_rng(13)
    nk, nq = 2500, 700
    rows = ref.mask([nk] + [0] * 3 + [1] * 600 + [700] + [3] * (nq - 605), nk, rng)
    for i in range(4, nq):
        if 7 not in rows[i]:
            rows[i][0] = 7
    q, k, v, dout = (_rand(rng, s, dtype) for s in ((nq, 2, 64), (nk, 1, 64), (nk, 1, 64),
                                                    (nq, 2, 64)))
    _check_both(rows, q, k, v, dout, nk, 0.125)


@pytest.mark.parametrize("dtype,hkv", [(BF16, 2), (F16, 1), (F16, 8), (F32, 2), (F32, 8)], ids=str)
def test_long_columns_and_head_counts(dtype, hkv):
    """2500 rows on 100 columns: blocks of columns that are cut finer for few
    key heads than for many."""
    rng = np.random.default_rng(hkv)
    rows, q, k, v, dout = _case(rng, dtype, 16, hkv, hkv, nk=100, lengths=[30] * 2500)
    _check_both(rows, q, k, v, dout, 100, 0.25)


def test_many_entries():
    """33 million entries, more than the plan carves its buffers out of one
    allocation for: every row sees every key, so sums over the dense product
    give the results."""
    api = _api()
    n, d = 5760, 8
    from spgemm_irregular_matrices_amd import binding
    rowptr = torch.arange(n + 1, device="cuda") * n
    col = torch.arange(n, device="cuda", dtype=torch.int32).repeat(n)
    rng = np.random.default_rng(26)
    q, k, v, dout = (_rand(rng, (n, 1, d), F32) for _ in range(4))
    with api.AttentionPlan(binding.DeviceCSR(n, n, rowptr, col, None), backward=True) as plan:
        out, lse = plan.forward(q, k, v, scale=0.3)
        grads = plan.backward(dout, q, k, v, out, lse, scale=0.3)
    Q, K, V, D = (x[:, 0].double().cpu() for x in (q, k, v, dout))
    s = 0.3 * Q @ K.T
    p = torch.softmax(s, 1)
    O = p @ V
    dp = D @ V.T
    ds = p * (dp - (D * O).sum(1, keepdim=True))
    # sums of 5760 terms in floats, each with a weight off by a few roundings:
    # (5760 + 64) * 2^-24 of the sums of magnitudes
    f = 6000 * 2.0 ** -24
    mag = p * (dp.abs() + D.abs() @ V.abs().T)
    for got, want, size in ((out, O, p @ V.abs()), (lse[..., None], torch.logsumexp(s, 1)[:, None],
                             torch.full((n, 1), 20.0)),
                            (grads[0], 0.3 * ds @ K, 0.3 * mag @ K.abs()),
                            (grads[1], 0.3 * ds.T @ Q, 0.3 * mag.T @ Q.abs()),
                            (grads[2], p.T @ D, p.T @ D.abs())):
        assert ((got[:, 0].double().cpu() - want).abs() <= f * size).all()


@pytest.mark.parametrize("nq,nk", [(0, 5), (5, 0), (0, 0), (1, 1)])
def test_empty_shapes(nq, nk):
    api = _api()
    rng = np.random.default_rng(14)
    rows = [np.arange(min(nk, 1)) for _ in range(nq)]
    q, k, v, dout = (_rand(rng, s, BF16) for s in ((nq, 2, 64), (nk, 2, 64), (nk, 2, 64),
                                                   (nq, 2, 64)))
    with api.AttentionPlan(ref.csr(rows, nk), backward=True) as plan:
        out, lse = plan.forward(q, k, v)
        dq, dk, dv = plan.backward(dout, q, k, v, out, lse)
    if nq and nk:
        assert torch.equal(out, v) and torch.equal(dv, dout)
    else:
        assert not out.any() and (lse == -float("inf")).all()
        assert not dq.any() and not dk.any() and not dv.any()


def test_extreme_scores():
    """Scores around 3e4 and -3e4: only differences to the row's largest enter exp."""
    rng = np.random.default_rng(15)
    rows, q, k, v, dout = _case(rng, BF16, 64, 2, 1)
    _check_both(rows, q * 64, k * 64, v, dout, 301, 1.0)


def test_infinite_keys_and_values_in_seen_places():
    """-inf scores weigh nothing; a row of nothing else counts as empty."""
    api = _api()
    rng = np.random.default_rng(16)
    rows = [np.array([0, 1, 2]), np.array([1]), np.array([2, 0])]
    q, k, v, dout = (_rand(rng, s, BF16) for s in ((3, 1, 64), (3, 1, 64), (3, 1, 64), (3, 1, 64)))
    q.fill_(1.0)
    k[1, 0, 5] = -float("inf")
    with api.AttentionPlan(ref.csr(rows, 3), backward=True) as plan:
        out, lse = plan.forward(q, k, v)
        assert torch.isfinite(out).all()
        assert lse[1, 0] == -float("inf") and not out[1].any()
        without = [np.array([0, 2]), np.array([], dtype=int), np.array([2, 0])]
        o, l, oe, le = ref.forward(ref.f64(q), np.nan_to_num(ref.f64(k), neginf=0), ref.f64(v),
                                   without, 0.125, BF16)
        ref.check(out, o, oe, "out")
        ref.check(lse, l, le, "lse")


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("wild", [float("nan"), float("inf")])
def test_gradients_of_wild_rows_stay_with_their_keys(dtype, wild):
    """NaN or infinities in one row's q and dout reach only that row and the
    keys it stores, not the neighbouring keys that share work with them."""
    api = _api()
    rng = np.random.default_rng(25)
    rows = ref.mask([40, 3, 40, 40, 2, 40], 48, rng)
    q, k, v, dout = (_rand(rng, s, dtype) for s in ((6, 4, 64), (48, 2, 64), (48, 2, 64), (6, 4, 64)))
    with api.AttentionPlan(ref.csr(rows, 48), backward=True) as plan:
        out, lse = plan.forward(q, k, v)
        clean = plan.backward(dout, q, k, v, out, lse)
        q[1], dout[4] = wild, wild
        out, lse = plan.forward(q, k, v)
        assert not torch.isfinite(out[1].float()).any()
        dq, dk, dv = plan.backward(dout, q, k, v, out, lse)
    mine = np.union1d(rows[1], rows[4])
    rest = torch.from_numpy(np.setdiff1d(np.arange(48), mine)).cuda()
    assert torch.equal(dk[rest], clean[1][rest]) and torch.equal(dv[rest], clean[2][rest])
    for i in (0, 2, 3, 5):
        assert torch.equal(dq[i], clean[0][i])
    assert not torch.isfinite(dk[torch.from_numpy(rows[1]).cuda()].float()).any()
    assert not torch.isfinite(dv[torch.from_numpy(rows[4]).cuda()].float()).any()


@pytest.mark.parametrize("amount", [1e-6, 1.0, 3e4])
def test_half_precision_gradients_of_any_size(amount):
    """Score gradients below and above what half precision holds."""
    rng = np.random.default_rng(17)
    rows, q, k, v, dout = _case(rng, F16, 64, 4, 2)
    small = 1e-2 if amount > 1 else 1.0
    q, k = (q.float() * small).half(), (k.float() * small).half()
    _check_both(rows, q, k, v, (dout.float() * amount).clamp(-6e4, 6e4).half(), 301, 1e-3)


def test_half_precision_many_small_weights():
    """5000 equal weights: each is below half precision's normal range."""
    rng = np.random.default_rng(18)
    nk = 5000
    rows = [np.arange(nk), np.arange(0, nk, 2)]
    q = torch.zeros(2, 2, 64, dtype=F16, device="cuda")
    k, v, dout = (_rand(rng, s, F16) for s in ((nk, 1, 64), (nk, 1, 64), (2, 2, 64)))
    v = v.abs()
    _check_both(rows, q, k, v, dout, nk, 0.125)


@pytest.mark.parametrize("layout", ["fused", "head_major", "broadcast", "gaps"])
def test_strides(layout):
    rng = np.random.default_rng(19)
    api = _api()
    n, hq, hkv, d = 70, 4, 2, 64
    rows = ref.mask(rng.integers(0, 70, n), n, rng)
    q, k, v, dout = (_rand(rng, s, BF16) for s in ((n, hq, d), (n, hkv, d), (n, hkv, d), (n, hq, d)))
    outs = {}
    if layout == "fused":
        qkv = torch.cat([q, k, v], 1)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        grad = torch.full_like(qkv, float("nan"))
        outs = dict(dq=grad[:, :hq], dk=grad[:, hq:hq + hkv], dv=grad[:, hq + hkv:])
    elif layout == "head_major":
        q, k, v, dout = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v, dout))
        outs = dict(dq=torch.empty(hq, n, d, dtype=BF16, device="cuda").transpose(0, 1))
    elif layout == "broadcast":
        k = k[:, :1].expand(-1, hkv, -1)
        dout = dout[:1].expand(n, -1, -1)
    else:
        q, k, v, dout = (torch.nn.functional.pad(x, (0, 24), value=float("nan"))[..., :d]
                         for x in (q, k, v, dout))
    with api.AttentionPlan(ref.csr(rows, n), backward=True) as plan:
        out, lse = plan.forward(q, k, v)
        got = plan.backward(dout, q, k, v, out, lse, **outs)
    a = [ref.f64(x) for x in (q, k, v)]
    o, l, oe, le = ref.forward(*a, rows, d ** -0.5, BF16)
    ref.check(out, o, oe, "out")
    want, err = ref.backward(*a, ref.f64(out), ref.f64(lse), ref.f64(dout), rows, d ** -0.5, BF16)
    for name, x, w, e in zip(("dq", "dk", "dv"), got, want, err):
        ref.check(x, w, e, name)


def test_offsets_past_32_bits():
    """Keys and values 96 KB apart, so that most lie past 4 GiB."""
    api = _api()
    rng = np.random.default_rng(20)
    nk, step, d = 70000, 49152, 64
    room = torch.empty(nk * step, dtype=BF16, device="cuda")
    k = room.as_strided((nk, 1, d), (step, d, 1))
    v = room.as_strided((nk, 1, d), (step, d, 1), 1024)
    rows = [np.array([0, 69999, 50000, 33333]), np.arange(69000, 69100)]
    rows += [np.array([69999])] * 3
    used = torch.from_numpy(np.unique(np.concatenate(rows))).cuda()
    k[used] = _rand(rng, (len(used), 1, d), BF16)
    v[used] = _rand(rng, (len(used), 1, d), BF16)
    q, dout = _rand(rng, (5, 2, d), BF16), _rand(rng, (5, 2, d), BF16)
    at = used.cpu().numpy()
    near = [np.searchsorted(at, r) for r in rows]
    with api.AttentionPlan(ref.csr(rows, nk), backward=True) as plan:
        out, lse = plan.forward(q, k, v)
        dq, dk, dv = plan.backward(dout, q, k, v, out, lse)
    a = [ref.f64(x) for x in (q, k[used], v[used])]
    o, l, oe, le = ref.forward(*a, near, 0.125, BF16)
    ref.check(out, o, oe, "out")
    want, err = ref.backward(*a, ref.f64(out), ref.f64(lse), ref.f64(dout), near, 0.125, BF16)
    for name, x, w, e in zip(("dq", "dk", "dv"), (dq, dk[used], dv[used]), want, err):
        ref.check(x, w, e, name)
    rest = torch.ones(nk, dtype=torch.bool, device="cuda")
    rest[used] = False
    assert not dk[rest].any() and not dv[rest].any()


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("d", [40, 64, 128, 200, 256])
def test_only_keys_have_no_gradient(dtype, d):
    """A row with one key: o is its value, and dq and dk are 0, to the last bit."""
    rng = np.random.default_rng(d)
    nq, nk = 37, 50
    q, dout = (_rand(rng, (nq, 4, d), dtype) for _ in range(2))
    k, v = (_rand(rng, (nk, 2, d), dtype) for _ in range(2))
    rows = [np.array([rng.integers(nk)]) for _ in range(nq)]
    api = _api()
    with api.AttentionPlan(ref.csr(rows, nk), backward=True) as plan:
        out, lse = plan.forward(q, k, v)
        dq, dk, dv = plan.backward(dout, q, k, v, out, lse)
    seen = torch.from_numpy(np.concatenate(rows)).cuda()
    assert torch.equal(out, v[seen].repeat_interleave(2, 1))
    assert not dq.any() and not dk.any()
    assert dv[seen].any()


def test_same_bits_every_time():
    api = _api()
    rng = np.random.default_rng(21)
    rows, q, k, v, dout = _case(rng, BF16, 128, 8, 2, nk=900, lengths=LENGTHS * 6 + [900] * 3)
    k, v = torch.nan_to_num(k), torch.nan_to_num(v, posinf=0)
    seen = []
    for _ in range(3):
        with api.AttentionPlan(ref.csr(rows, 900), backward=True) as plan:
            out, lse = plan.forward(q, k, v)
            seen.append((out, lse, *plan.backward(dout, q, k, v, out, lse)))
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))


def test_gradient_against_differences():
    """(f(x + t y) - f(x - t y)) / 2t of f = sum(out * dout), in floats.

    The third derivative's term: t^2 / 6 * |f'''|, which for t = 1/64 and
    directions of entries about 1 is under 1e-3 of the derivative's scale; the
    differences' rounding: outputs of about 1 with relative error 1e-6 in
    sums over 4e3 entries of random sign, over 2t, is under 1e-2 absolute."""
    api = _api()
    rng = np.random.default_rng(22)
    n, d = 40, 32
    rows = ref.mask(rng.integers(0, n, n), n, rng)
    q, k, v, dout = (_rand(rng, s, F32) for s in ((n, 4, d), (n, 2, d), (n, 2, d), (n, 4, d)))
    with api.AttentionPlan(ref.csr(rows, n), backward=True) as plan:
        out, lse = plan.forward(q, k, v)
        grads = plan.backward(dout, q, k, v, out, lse)
        for at in range(3):
            y = _rand(rng, (q, k, v)[at].shape, F32)
            f = []
            for t in (1 / 64, -1 / 64):
                x = [q, k, v]
                x[at] = x[at] + t * y
                f.append((plan.forward(*x)[0].double() * dout.double()).sum().item())
            slope = (f[0] - f[1]) * 32
            want = (grads[at].double() * y.double()).sum().item()
            size = (grads[at].double() * y.double()).abs().sum().item()
            assert abs(slope - want) <= 1e-3 * size + 1e-2, (at, slope, want, size)


def test_other_stream_and_graph():
    """A captured forward and backward, replayed between eager work on new inputs."""
    api = _api()
    rng = np.random.default_rng(23)
    rows, q, k, v, dout = _case(rng, BF16, 64, 4, 2, lengths=LENGTHS + [301])
    k, v = torch.nan_to_num(k), torch.nan_to_num(v, posinf=0)
    with api.AttentionPlan(ref.csr(rows, 301), backward=True) as plan:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out, lse = plan.forward(q, k, v, stream=side)
        grads = plan.backward(dout, q, k, v, out, lse, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        eager = [x.clone() for x in (out, lse, *grads)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, l = plan.forward(q, k, v)
            g = plan.backward(dout, q, k, v, o, l)
        for step in range(4):
            fresh = _rand(rng, q.shape, BF16)
            q.copy_(fresh)
            graph.replay()
            eager = plan.forward(q, k, v)
            eager = (*eager, *plan.backward(dout, q, k, v, *eager))
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((o, l, *g), eager)), step


def test_two_plans_and_streams_at_once():
    api = _api()
    rng = np.random.default_rng(24)
    rows, q, k, v, dout = _case(rng, BF16, 64, 4, 2, lengths=LENGTHS * 20)
    k, v = torch.nan_to_num(k), torch.nan_to_num(v, posinf=0)
    with api.AttentionPlan(ref.csr(rows, 301), backward=True) as plan:
        want = plan.forward(q, k, v)
        want = (*want, *plan.backward(dout, q, k, v, *want))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = []
        for s in streams:
            o, l = plan.forward(q, k, v, stream=s)
            got.append((o, l, *plan.backward(dout, q, k, v, o, l, stream=s)))
        torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


# ---------------------------------------------------------------- paged
def _paged_case(rng, dtype, d, hq, hkv, page, seqs, pad=3, layout="slots"):
    """seqs: (cached tokens, new ones among them). The cache holds NaN and
    infinities wherever no sequence's token lies."""
    count = [(n + page - 1) // page for n, _ in seqs]
    pool = sum(count) + 2
    order = rng.permutation(pool)[:sum(count)]
    shape = (pool, hkv, page, d) if layout == "heads" else (pool, page, hkv, d)
    kc, vc = torch.full(shape, float("nan"), dtype=dtype), torch.full(shape, float("inf"), dtype=dtype)
    if layout == "heads":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    keys = [torch.from_numpy(rng.standard_normal((2, n, hkv, d))).to(dtype) for n, _ in seqs]
    rowptr = np.concatenate([[0], np.cumsum(count)]).astype(np.int64)
    for s, (n, _) in enumerate(seqs):
        for j in range(n):
            kc[order[rowptr[s] + j // page], j % page] = keys[s][0, j]
            vc[order[rowptr[s] + j // page], j % page] = keys[s][1, j]
    start = np.concatenate([[0], np.cumsum([m for _, m in seqs])]).astype(np.int64)
    tokens = int(start[-1]) + pad
    q = torch.from_numpy(rng.standard_normal((tokens, hq, d))).to(dtype).cuda()
    from spgemm_irregular_matrices_amd import binding
    table = binding.DeviceCSR(len(seqs), pool, torch.from_numpy(rowptr).cuda(),
                              torch.from_numpy(order.astype(np.int32)).cuda(), None)
    return dict(q=q, k=kc.cuda() if layout != "heads" else kc.transpose(1, 2).contiguous().cuda().transpose(1, 2),
                v=vc.cuda() if layout != "heads" else vc.transpose(1, 2).contiguous().cuda().transpose(1, 2),
                table=table, q_rowptr=torch.from_numpy(start).cuda(),
                lengths=torch.tensor([n for n, _ in seqs], dtype=torch.int64).cuda(),
                max_q=max(m for _, m in seqs), max_len=max(n for n, _ in seqs), keys=keys)


def _paged_run(c, **more):
    return _api().paged_attention(c["q"], c["k"], c["v"], c["table"], c["q_rowptr"], c["lengths"],
                                  **{"max_q": c["max_q"], "max_len": c["max_len"], **more})


def _paged_check(c, seqs, scale, out, lse, skip=()):
    dtype = c["q"].dtype
    at = 0
    for s, (n, m) in enumerate(seqs):
        if s not in skip:
            rows = [np.arange(n - m + t + 1) for t in range(m)]
            kk, vv = ref.f64(c["keys"][s][0]), ref.f64(c["keys"][s][1])
            o, l, oe, le = ref.forward(ref.f64(c["q"][at:at + m]), kk, vv, rows, scale, dtype)
            ref.check(out[at:at + m], o, oe, f"out of sequence {s}")
            ref.check(lse[at:at + m], l, le, f"lse of sequence {s}")
        at += m


SEQS = [(1, 1), (33, 1), (40, 7), (5, 5), (0, 0), (130, 2), (200, 33), (64, 64)]


@pytest.mark.parametrize("dtype,d,hq,hkv,page", [
    (BF16, 64, 4, 2, 16), (BF16, 128, 8, 1, 1), (F16, 64, 7, 1, 24), (F32, 64, 3, 3, 7),
    (BF16, 40, 2, 2, 64), (F16, 256, 16, 1, 32), (F32, 136, 4, 2, 128), (BF16, 128, 20, 1, 5),
    (F32, 4, 1, 1, 3)])
def test_paged(dtype, d, hq, hkv, page):
    rng = np.random.default_rng(hq * 1000 + page)
    c = _paged_case(rng, dtype, d, hq, hkv, page, SEQS)
    keep = torch.full_like(c["q"], 7.0)
    lse = torch.full(c["q"].shape[:2], 9.0, device="cuda")
    out, lse = _paged_run(c, out=keep, lse=lse, scale=d ** -0.5)
    _paged_check(c, SEQS, d ** -0.5, out, lse)
    assert (out[-3:] == 7.0).all() and (lse[-3:] == 9.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("hq,hkv", [(8, 1), (2, 2), (20, 1)])
def test_paged_single_tokens(dtype, hq, hkv):
    """The next token of sequences of one to 700 cached ones, pieces joined."""
    rng = np.random.default_rng(31)
    seqs = [(n, 1) for n in (1, 2, 31, 32, 33, 63, 64, 65, 500, 700)]
    c = _paged_case(rng, dtype, 64, hq, hkv, 16, seqs)
    out, lse = _paged_run(c)
    _paged_check(c, seqs, 0.125, out, lse)


def test_paged_head_major_cache():
    rng = np.random.default_rng(32)
    c = _paged_case(rng, BF16, 64, 4, 2, 16, SEQS, layout="heads")
    out, lse = _paged_run(c)
    _paged_check(c, SEQS, 0.125, out, lse)


def test_paged_long_chunk():
    rng = np.random.default_rng(33)
    seqs = [(300, 150), (260, 260), (129, 1)]
    c = _paged_case(rng, BF16, 128, 8, 2, 16, seqs)
    out, lse = _paged_run(c)
    _paged_check(c, seqs, 128 ** -0.5, out, lse)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("wild", [float("nan"), float("inf"), -float("inf")])
def test_paged_later_tokens_reach_nothing(dtype, wild):
    """NaN or infinities in a later token's key and value leave earlier tokens alone."""
    rng = np.random.default_rng(34)
    seqs = [(50, 20), (9, 9)]
    c = _paged_case(rng, dtype, 64, 4, 2, 16, seqs)
    clean_out, clean_lse = _paged_run(c)
    first = int(c["table"].rowptr[0])
    page = int(c["table"].col[first + 45 // 16])
    c["k"][page, 45 % 16] = wild
    c["v"][page, 45 % 16] = wild
    out, lse = _paged_run(c)
    before = 45 - 30  # tokens of the chunk that do not see cached token 45
    assert torch.equal(out[:before], clean_out[:before])
    assert torch.equal(lse[:before], clean_lse[:before])
    assert torch.equal(out[20:29], clean_out[20:29])
    assert not torch.isfinite(out[before:20]).all(2).any()


@pytest.mark.parametrize("new", [8, 24, 120])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("d", [64, 128, 200])
def test_paged_chunk_sizes(dtype, d, new):
    """Chunks of 16 to 240 rows to a key head, in the tiles of single wavefronts
    and of work groups; then a wild key and value that only later tokens see."""
    rng = np.random.default_rng(d + new)
    seqs = [(40 + new, new), (new, new), (310, max(1, new // 3)), (3, 1)]
    c = _paged_case(rng, dtype, d, 4, 2, 16, seqs)
    clean = _paged_run(c)
    _paged_check(c, seqs, d ** -0.5, *clean)
    at = 40 + new // 2  # seen by the first sequence's tokens from new // 2 on
    page = int(c["table"].col[at // 16])
    c["k"][page, at % 16], c["v"][page, at % 16] = float("nan"), float("inf")
    got = _paged_run(c)
    sees = torch.zeros(len(c["q"]), dtype=torch.bool, device="cuda")
    sees[new // 2:new] = True
    tokens = sum(m for _, m in seqs)
    for a, b in zip(got, clean):
        assert torch.equal(a[:tokens][~sees[:tokens]], b[:tokens][~sees[:tokens]])
    assert not torch.isfinite(got[0][sees].float()).any()
    assert not torch.isfinite(got[1][sees]).any()


def test_paged_equals_lower_triangular_mask():
    """Used together: a text read in chunks over the cache gives what one call
    over a lower triangular mask gives, to the roundings of the two."""
    api = _api()
    rng = np.random.default_rng(35)
    n, hq, hkv, d, page = 150, 4, 2, 64, 16
    c = _paged_case(rng, BF16, d, hq, hkv, page, [(n, n)], pad=0)
    kk, vv = c["keys"][0].cuda()
    rows = [np.arange(i + 1) for i in range(n)]
    with api.AttentionPlan(ref.csr(rows, n), backward=True) as plan:
        out, lse = plan.forward(c["q"], kk, vv)
    o, l, oe, le = ref.forward(ref.f64(c["q"]), ref.f64(kk), ref.f64(vv), rows, 0.125, BF16)
    ref.check(out, o, oe, "out")
    at = 0
    for step in (1, 64, 3, 50, 1, 31):
        sub = dict(c, q=c["q"][at:at + step], max_q=step, max_len=at + step,
                   q_rowptr=torch.tensor([0, step]).cuda(), lengths=torch.tensor([at + step]).cuda())
        po, pl = _paged_run(sub)
        ref.check(po, o[at:at + step], oe[at:at + step], "chunk out")
        ref.check(pl, l[at:at + step], le[at:at + step], "chunk lse")
        at += step
    assert at == n


def test_paged_bad_batches_give_nan():
    """Sequences that break the rules get NaN; their neighbours do not notice."""
    rng = np.random.default_rng(36)
    seqs = [(40, 2), (70, 3), (33, 1), (20, 2)]
    c = _paged_case(rng, BF16, 64, 4, 2, 16, seqs)

    def expect(bad, **changed):
        out, lse = _paged_run({**c, **changed}, out=torch.zeros_like(c["q"]))
        _paged_check(c, seqs, 0.125, out, lse, skip=(bad,))
        at = sum(m for _, m in seqs[:bad])
        assert torch.isnan(out[at:at + seqs[bad][1]]).all()
        assert torch.isnan(lse[at:at + seqs[bad][1]]).all()
        assert not out[-3:].any()

    from spgemm_irregular_matrices_amd import binding
    t = c["table"]
    for value in (-1, t.ncols, 2 ** 31 - 1, -2 ** 31):
        col = t.col.clone()
        col[int(t.rowptr[1])] = value
        expect(1, table=binding.DeviceCSR(t.nrows, t.ncols, t.rowptr, col, None))
    for length in (2, -1, 81, 10 ** 12):  # below its new tokens, none, past its pages, past max_len
        lengths = c["lengths"].clone()
        lengths[1] = length
        expect(1, lengths=lengths)
    expect(1, max_len=69)
    rowptr = t.rowptr.clone()
    rowptr[-1] = 10 ** 9  # past the table's room
    expect(3, table=binding.DeviceCSR(t.nrows, t.ncols, rowptr, t.col, None))


def test_paged_graph_follows_the_batch():
    """A captured step, replayed as the texts grow, between eager calls."""
    rng = np.random.default_rng(37)
    seqs = [(100, 1), (37, 1), (64, 1)]
    c = _paged_case(rng, BF16, 64, 8, 2, 16, seqs, pad=1)
    lengths = c["lengths"].clone()
    c["lengths"] = torch.tensor([3, 2, 1]).cuda()
    graph = torch.cuda.CUDAGraph()
    _paged_run(c)
    with torch.cuda.graph(graph):
        out, lse = _paged_run(c)
    for step in range(4):
        c["lengths"].copy_(lengths * (step + 1) // 4)
        c["q"].copy_(_rand(rng, c["q"].shape, BF16))
        graph.replay()
        o, l = _paged_run(c)
        torch.cuda.synchronize()
        assert torch.equal(out[:3], o[:3]) and torch.equal(lse[:3], l[:3]), step
    _paged_check(c, seqs, 0.125, out, lse)


def test_paged_without_work():
    rng = np.random.default_rng(38)
    c = _paged_case(rng, BF16, 64, 2, 1, 16, [(5, 1)], pad=0)
    out = torch.full_like(c["q"], 3.0)
    empty = dict(c, q_rowptr=torch.tensor([0, 0]).cuda())
    _paged_run(empty, out=out)
    _paged_run(c, out=out, max_q=0)
    from spgemm_irregular_matrices_amd import binding
    none = binding.DeviceCSR(0, c["table"].ncols, torch.zeros(1, dtype=torch.int64).cuda(),
                             torch.zeros(0, dtype=torch.int32).cuda(), None)
    _paged_run(dict(c, table=none, q_rowptr=torch.zeros(1, dtype=torch.int64).cuda(),
                    lengths=torch.zeros(0, dtype=torch.int64).cuda()), out=out)
    assert (out == 3.0).all()


# ---------------------------------------------------------------- refusals
def test_plan_refusals():
    api = _api()
    from spgemm_irregular_matrices_amd import binding
    good = ref.csr([np.array([0, 2]), np.array([1])], 3)

    def code(m, **more):
        with pytest.raises(binding.SpgemmError) as e:
            api.AttentionPlan(m, **more)
        return e.value.code

    D = binding.DeviceCSR
    i64 = lambda *x: torch.tensor(x, dtype=torch.int64).cuda()  # noqa: E731
    for col in (3, -1):
        assert code(D(2, 3, good.rowptr, torch.tensor([0, 2, col], dtype=torch.int32).cuda(), None)) == -3
    for rp in (i64(0, 2, 2), i64(1, 2, 3), i64(0, 4, 3), i64(0, -1, 3)):
        assert code(D(2, 3, rp, good.col, None)) == -3
    assert code(D(2, 2 ** 31, good.rowptr, good.col, None)) == -4
    for bad in (D(2, 3, good.rowptr.int(), good.col, None), D(3, 3, good.rowptr, good.col, None),
                D(2, 3, good.rowptr, good.col.long(), None), D(2, 3, good.rowptr.cpu(), good.col, None)):
        with pytest.raises(ValueError):
            api.AttentionPlan(bad)
    plan = api.AttentionPlan(good)
    q = torch.zeros(2, 2, 64, dtype=BF16, device="cuda")
    k = torch.zeros(3, 1, 64, dtype=BF16, device="cuda")
    out, lse = plan.forward(q, k, k)
    with pytest.raises(binding.SpgemmError) as e:
        plan.backward(q, q, k, k, out, lse)
    assert e.value.code == -8  # made without backward
    plan.close()
    with pytest.raises(ValueError):
        plan.forward(q, k, k)


def test_tensor_refusals():
    api = _api()
    from spgemm_irregular_matrices_amd import binding
    plan = api.AttentionPlan(ref.csr([np.array([0, 2]), np.array([1])], 3), backward=True)
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    q, k = z(2, 4, 64), z(3, 2, 64)
    out, lse = plan.forward(q, k, k)
    for bad in ((z(3, 4, 64), k, k), (q, z(2, 2, 64), k), (q, k, z(3, 1, 64)), (q, k, z(3, 2, 32)),
                (q, k.float(), k), (q.double(), k.double(), k.double()), (q, k, k.cpu()),
                (q[0], k, k), (q, z(3, 64, 2).transpose(1, 2), k)):
        with pytest.raises(ValueError):
            plan.forward(*bad)

    def code(*args, **more):
        with pytest.raises(binding.SpgemmError) as e:
            plan.forward(*args, **more)
        return e.value.code

    assert code(q, z(3, 3, 64), z(3, 3, 64)) == -1            # 4 heads over 3
    assert code(z(2, 4, 12), z(3, 2, 12), z(3, 2, 12)) == -1  # rows of 24 bytes
    assert code(z(2, 4, 264), z(3, 2, 264), z(3, 2, 264)) == -1
    assert code(q, k, k, scale=float("nan")) == -1
    assert code(z(2, 4, 68)[..., :64], k, k) == -1            # a stride of 136 bytes
    odd = z(2 * 4 * 64 + 4)[4:].view(2, 4, 64)
    assert code(odd, k, k) == -1                              # an address of 8 bytes
    assert code(q, k, k, out=z(2, 1, 64).expand(2, 4, 64)) == -1  # rows that overlap
    with pytest.raises(ValueError):
        plan.forward(q, k, k, lse=z(2, 4))
    with pytest.raises(ValueError):
        plan.backward(out, q, k, k, out, lse.double())
    # a workspace that is too small, through the C call
    lib = api.load()
    long = api.AttentionPlan(ref.csr([np.arange(1000)], 1000))
    big = z(1000, 1, 64)
    one = z(1, 1, 64)
    d = api.Desc(0, 1, 1, 64, 1.0)
    need = ctypes.c_int64()
    assert lib.spgemm_attention_workspace(long._h, ctypes.byref(d), 0, ctypes.byref(need)) == 0
    assert need.value > 0
    space = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    r, kr = api.Rows(one.data_ptr(), 64, 64), api.Rows(big.data_ptr(), 64, 64)
    args = [ctypes.byref(x) for x in (d, r, kr, kr, r)]
    assert lib.spgemm_attention_forward(long._h, *args, None, space.data_ptr(), need.value - 1, None) == -1
    assert lib.spgemm_attention_forward(long._h, *args, None, None, need.value, None) == -1
    assert lib.spgemm_attention_forward(long._h, *args, None, space.data_ptr(), need.value, None) == 0
    torch.cuda.synchronize()
    plan.close()
    long.close()


def test_offsets_that_do_not_fit_are_refused():
    """Rows so far apart that no power of two fits their offsets into 32 bits
    (checked before any kernel runs: nothing of them is read)."""
    api = _api()
    lib = api.load()
    plan = api.AttentionPlan(ref.csr([np.array([0, 2]), np.array([1])], 3), backward=True)
    one = torch.zeros(8, 64, dtype=BF16, device="cuda")
    far = (1 << 36) + 8
    d = api.Desc(0, 1, 1, 64, 1.0)
    near, wide = api.Rows(one.data_ptr(), 64, 64), api.Rows(one.data_ptr(), far, 64)
    lse = torch.zeros(2, device="cuda")
    space = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    at = lambda *x: [ctypes.byref(y) for y in x]  # noqa: E731
    tail = (space.data_ptr(), 1 << 16, None)
    assert lib.spgemm_attention_forward(plan._h, *at(d, near, wide, near, near), None, *tail) == -4
    assert lib.spgemm_attention_forward(plan._h, *at(d, near, near, wide, near), None, *tail) == -4
    grads = at(near, near, near, near)
    for q, dout in ((wide, near), (near, wide)):
        assert lib.spgemm_attention_backward(plan._h, *at(d, q, near, near, near), lse.data_ptr(),
                                             ctypes.byref(dout), *grads[:3], *tail) == -4
    assert lib.spgemm_attention_forward(plan._h, *at(d, near, near, near, near), None, *tail) == 0
    torch.cuda.synchronize()
    plan.close()


def test_paged_refusals():
    rng = np.random.default_rng(39)
    c = _paged_case(rng, BF16, 64, 4, 2, 16, [(20, 1), (5, 2)])
    bad = [dict(lengths=c["lengths"].int()), dict(q_rowptr=c["q_rowptr"][:-1]),
           dict(k=c["k"].float()), dict(v=c["v"][:, :8]), dict(q=c["q"][0]),
           dict(k=c["k"][1:], v=c["v"][1:])]
    for b in bad:
        with pytest.raises(ValueError):
            _paged_run({**c, **b})
    from spgemm_irregular_matrices_amd import binding
    for more in (dict(max_len=-1), dict(max_q=-1), dict(scale=float("inf"))):
        with pytest.raises(binding.SpgemmError) as e:
            _paged_run(c, **more)
        assert e.value.code == -1
    with pytest.raises(binding.SpgemmError) as e:
        _paged_run(c, max_len=2 ** 31)
    assert e.value.code == -4
