"""Attention on the GPU where its formulas meet the ends of the types: against
the definition in 64 bits, with bounds derived beside each test."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import attention_ref as ref  # noqa: E402
from tests.test_gpu_attention import BF16, F16, F32, _api, _gpu, _paged_case, _paged_run, _rand  # noqa: E402, F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- scores of any size
def _signs(rng, shape, amount, dtype):
    """Entries of +-amount, a power of two: every dot product is a whole multiple of a power of
    two below 2^24 such units, so that scores are exact in floats and in any order of summing."""
    return torch.from_numpy(rng.choice([-amount, amount], shape)).to(dtype).cuda()


def _one_hot(q, k, v, rows):
    """out and lse where the keys with a row's largest score, which differ from all others by
    2^7 and more, share all of the weight (another's is below e^-128); and a bound of out's error:
    equal weights of 1, n of them summed and divided in floats, then one rounding to the type."""
    (nq, H, _), G = q.shape, q.shape[1] // k.shape[1]
    out, err, lse = np.zeros_like(q), np.zeros_like(q), np.full((nq, H), -np.inf)
    for i, cols in enumerate(rows):
        for h in range(H if len(cols) else 0):
            s = k[cols, h // G] @ q[i, h]
            top = np.asarray(cols)[s == s.max()]
            vv = v[top, h // G]
            out[i, h], lse[i, h] = vv.mean(0), s.max() + np.log(len(top))
            err[i, h] = (len(top) + 4) * ref.E * np.abs(vv).mean(0)
    return out, lse, err


def _check_one_hot(out, lse, want, dtype, ones):
    o, l, err = want
    u = ref.U[dtype]
    ref.check(out, o, err + u * np.abs(o) + (2.0 ** -25 if dtype == F16 else 0), "out")
    ref.check(lse, l, 8 * ref.E * np.abs(l), "lse")  # maximum times factor, its way back, the sum
    assert np.array_equal(ref.f64(out)[ones], o[ones], equal_nan=True)  # one key: its value unchanged


SIZES = [(BF16, 2.0 ** 4), (BF16, 2.0 ** 9), (BF16, 2.0 ** 20), (BF16, 2.0 ** 50), (F16, 2.0 ** 4),
         (F16, 2.0 ** 6), (F16, 2.0 ** 10), (F16, 2.0 ** 12), (F16, 2.0 ** 15), (F32, 2.0 ** 4), (F32, 2.0 ** 20), (F32, 2.0 ** 50)]


@pytest.mark.parametrize("dtype,amount", SIZES, ids=str)
@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("order", ["ascending", "shuffled"])
def test_scores_of_any_size(dtype, amount, d, order):
    """The largest weight is 1 however large the scores are: what rounds their factor away must
    not enter the weights' exponents."""
    api = _api()
    rng = np.random.default_rng(d)
    rows = ref.mask([1, 1, 1, 1, 0, 5, 300, 40, 33, 1, 0, 0, 64, 65, 3, 2, 17], 300, rng)
    if order == "ascending":
        rows = [np.sort(r) for r in rows]
    ones = np.array([len(r) == 1 for r in rows])
    q, k = _signs(rng, (len(rows), 4, d), amount, dtype), _signs(rng, (300, 2, d), 8 * amount, dtype)
    # (half precision's 8 * 2^15 is infinite: rows of infinities of both signs, all NaN)
    v = _rand(rng, (300, 2, d), dtype)
    with api.AttentionPlan(ref.csr(rows, 300)) as plan:
        out, lse = plan.forward(q, k, v, scale=1.0)
    _check_one_hot(out, lse, _one_hot(*[ref.f64(x) for x in (q, k, v)], rows), dtype, ones)


@pytest.mark.parametrize("dtype,amount", SIZES, ids=str)
@pytest.mark.parametrize("d,new", [(64, 1), (64, 40), (128, 1), (128, 30), (200, 2), (200, 70)])
def test_paged_scores_of_any_size(dtype, amount, d, new):
    rng = np.random.default_rng(d + new)
    seqs = [(300 + new, new), (new, new), (1, 1)]
    c = _paged_case(rng, dtype, d, 4, 2, 16, seqs, pad=0)
    factor = 1 if dtype == F16 and amount > 2.0 ** 12 else 8
    c["q"] = _signs(rng, c["q"].shape, amount, dtype)
    t = c["table"]
    for s, (n, _) in enumerate(seqs):
        c["keys"][s][0] = _signs(rng, c["keys"][s][0].shape, factor * amount, dtype).cpu()
        for j in range(n):
            c["k"][int(t.col[int(t.rowptr[s]) + j // 16]), j % 16] = c["keys"][s][0][j].cuda()
    out, lse = _paged_run(c, scale=1.0)
    at = 0
    for s, (n, m) in enumerate(seqs):
        rows = [np.arange(n - m + i + 1) for i in range(m)]
        ones = np.array([len(r) == 1 for r in rows])
        want = _one_hot(*[ref.f64(x) for x in (c["q"][at:at + m], *c["keys"][s])], rows)
        _check_one_hot(out[at:at + m], lse[at:at + m], want, dtype, ones)
        at += m


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("amount", [1, 3, 8, 11, 16, 60, 200])
def test_only_keys_of_any_score(dtype, amount):
    """A row with one key gives its value unchanged: below 2^12 the maximum's rounding and that of its
    difference to the shift are up to 2^-13 each, so that the weight is off by up to 2^-12 log 2, under
    half a step of half precision and of the quotient; from there on it is 1."""
    api = _api()
    rng = np.random.default_rng(amount)
    n, d = 600, 64
    q, k, v = (_rand(rng, (n, h, d), dtype, s) for h, s in ((4, amount * 4), (2, amount * 4), (2, 1)))
    at = rng.permutation(n)
    with api.AttentionPlan(ref.csr([np.array([j]) for j in at], n)) as plan:
        out, _ = plan.forward(q, k, v, scale=0.4)
    assert torch.equal(out, v[torch.from_numpy(at).cuda()].repeat_interleave(2, 1))
    c = _paged_case(rng, dtype, d, 4, 2, 16, [(1, 1)] * 50)
    c["q"].mul_(amount * 4)
    c["k"].mul_(amount * 4)
    out, _ = _paged_run(c, scale=0.4)
    want = torch.stack([x[1, 0] for x in c["keys"]]).cuda().repeat_interleave(2, 1)
    assert torch.equal(out[:50], want)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("new", [3, 40])
def test_large_scores_leave_other_rows_alone(dtype, new):
    """Rows that share tiles with one of huge scores keep their bits."""
    api = _api()
    rng = np.random.default_rng(new)
    rows = [np.arange(max(0, i - 20), i + 1) for i in range(60)]
    q, k, v = (_rand(rng, s, dtype) for s in ((60, 4, 64), (60, 2, 64), (60, 2, 64)))
    c = _paged_case(rng, dtype, 64, 4, 2, 16, [(200, new)], pad=0)
    with api.AttentionPlan(ref.csr(rows, 60)) as plan:
        clean = plan.forward(q, k, v), _paged_run(c)
        q[1], c["q"][1] = q[1] * 2.0 ** 13, c["q"][1] * 2.0 ** 13
        got = plan.forward(q, k, v), _paged_run(c)
    for a, b in zip(clean, got):
        for x, y in zip(a, b):
            keep = torch.arange(len(x), device="cuda") != 1
            assert torch.equal(x[keep], y[keep]) and not torch.equal(x[1], y[1])
            assert torch.isfinite(y).all()


@pytest.mark.parametrize("dtype,amount", [x for x in SIZES if x != (F16, 2.0 ** 15)], ids=str)
@pytest.mark.parametrize("d", [64, 128, 200])
def test_gradients_of_scores_of_any_size(dtype, amount, d):
    """A weight is exp(s - lse) of two floats, so that of large scores its error passes 1; but it
    is at most 1. So |dv_j| <= sum_i |dout_i| (n terms summed in floats, one rounding to the type),
    and a row's only key has dS = p (dP - delta) = p * 0 = 0."""
    api = _api()
    rng = np.random.default_rng(d)
    rows = ref.mask([1, 1, 1, 1, 0, 5, 200, 40, 33, 0, 64, 65, 3, 2, 17], 250, rng)
    alone = np.arange(250, 254)  # keys 250 to 253: seen by one row each, which sees nothing else
    rows[:4] = [np.array([j]) for j in alone]
    q, k = _signs(rng, (len(rows), 4, d), amount, dtype), _signs(rng, (254, 2, d), 8 * amount, dtype)
    v, dout = _rand(rng, (254, 2, d), dtype), _rand(rng, (len(rows), 4, d), dtype)
    with api.AttentionPlan(ref.csr(rows, 254), backward=True) as plan:
        out, lse = plan.forward(q, k, v, scale=1.0)
        dq, dk, dv = plan.backward(dout, q, k, v, out, lse, scale=1.0)
    assert torch.isfinite(dv).all()
    for x in (dq, dk):
        # one key's dS k is up to |dP - delta| * 8 amount, in half precision 20 * 8 * 2^10 for
        # instance, past its largest of 65504: infinities are that type's results there
        assert not torch.isnan(x).any() and (dtype == F16 or torch.isfinite(x).all())
    assert not dq[:4].any() and not dk[250:].any()
    most = np.zeros(v.shape)
    for i, cols in enumerate(rows):
        for h in range(4):
            np.add.at(most[:, h // 2], cols, np.abs(ref.f64(dout)[i, h]))
    n = sum(len(r) for r in rows) * 2
    assert (np.abs(ref.f64(dv)) <= most * (1 + ref.U[dtype] + n * ref.E)).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=str)
@pytest.mark.parametrize("wild", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("new", [2, 40])
def test_scale_of_zero_keeps_wild_queries(dtype, wild, new):
    """0 times a score that is not a number is not a number: such a query's row is NaN (to a
    NaN sum belongs a NaN), and others are the mean of their values."""
    api = _api()
    rng = np.random.default_rng(new)
    rows = ref.mask([3, 17, 40, 33, 1, 2, 60, 5], 60, rng)
    q, k, v = (_rand(rng, s, dtype) for s in ((8, 4, 64), (60, 2, 64), (60, 2, 64)))
    c = _paged_case(rng, dtype, 64, 4, 2, 16, [(100, new)], pad=0)
    with api.AttentionPlan(ref.csr(rows, 60)) as plan:
        clean = plan.forward(q, k, v, scale=0.0), _paged_run(c, scale=0.0)
        q[1, 2, 5], c["q"][1, 2, 5] = wild, wild
        got = plan.forward(q, k, v, scale=0.0), _paged_run(c, scale=0.0)
    for a, b in zip(clean, got):
        for x, y in zip(a, b):
            keep = torch.ones(x.shape[:2], dtype=torch.bool, device="cuda")
            keep[1, 2] = False
            assert torch.equal(x[keep], y[keep]) and torch.isfinite(x).all()
            assert torch.isnan(y[1, 2]).all()


def test_a_function_of_autograd():
    """forward and backward in a user's autograd Function: leaves get the gradients of the calls."""
    api = _api()
    rng = np.random.default_rng(41)
    rows = [np.arange(max(0, i - 9), i + 1) for i in range(40)]
    q, k, v = (_rand(rng, s, F32) for s in ((40, 4, 64), (40, 2, 64), (40, 2, 64)))
    dout = _rand(rng, q.shape, F32)
    with api.AttentionPlan(ref.csr(rows, 40), backward=True) as plan:

        class Attention(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v):
                out, lse = plan.forward(q, k, v)
                ctx.save_for_backward(q, k, v, out, lse)
                return out

            @staticmethod
            def backward(ctx, dout):
                return plan.backward(dout.contiguous(), *ctx.saved_tensors)

        out, lse = plan.forward(q, k, v)
        want = plan.backward(2 * dout, q, k, v, out, lse)
        leaves = [x.clone().requires_grad_() for x in (q, k, v)]
        with pytest.raises(ValueError):
            plan.forward(*leaves)
        (2 * dout * Attention.apply(*leaves)).sum().backward()
    for x, g in zip(leaves, want):
        assert torch.equal(x.grad, g)
