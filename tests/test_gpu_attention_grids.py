"""Calls whose launches count more than 2^32 lanes along one axis of the grid."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from spgemm_irregular_matrices_amd import binding  # noqa: E402
from tests import attention_ref as ref  # noqa: E402
from tests.test_gpu_attention import BF16, _api, _gpu, _paged_case, _paged_check, _paged_run, _rand  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def _padded(c, seqs, count, tokens):
    """The batch with sequences without tokens up to `count`, and rows of no sequence up to `tokens`."""
    t, more = c["table"], count - len(seqs)
    pad = lambda x: torch.cat([x, x[-1:].expand(more)])  # noqa: E731
    q = torch.zeros(tokens, *c["q"].shape[1:], dtype=c["q"].dtype, device="cuda")
    q[:len(c["q"])] = c["q"]
    return dict(c, q=q, q_rowptr=pad(c["q_rowptr"]), lengths=pad(c["lengths"]),
                table=binding.DeviceCSR(count, t.ncols, pad(t.rowptr), t.col, None))


def test_paged_many_tiles():
    """Room for 4096 new tokens of 64 heads in each of 16384 sequences: 2^25 tiles of 128 rows."""
    rng = np.random.default_rng(61)
    seqs = [(70, 5), (300, 90), (33, 1)]
    c = _padded(_paged_case(rng, BF16, 8, 64, 1, 16, seqs), seqs, 16384, 4096)
    out, lse = _paged_run(c, max_q=4096, out=torch.full_like(c["q"], 7.0))
    _paged_check(c, seqs, 8 ** -0.5, out, lse)
    assert (out[96:] == 7).all()


def test_paged_many_sequences():
    """300000 sequences and 64 key heads, most without tokens: 4.8 million work groups."""
    rng = np.random.default_rng(65)
    seqs = [(70, 1), (128, 1), (33, 1), (100, 1)]
    c = _padded(_paged_case(rng, BF16, 8, 64, 64, 16, seqs), seqs, 300000, 7)
    out, lse = _paged_run(c, out=torch.full_like(c["q"], 7.0))
    _paged_check(c, seqs, 8 ** -0.5, out, lse)
    assert (out[4:] == 7).all()


def test_paged_join_of_many_rows():
    """2^20 + 3 rows of 64 heads, most of no sequence, and texts of two pieces."""
    rng = np.random.default_rng(62)
    seqs = [(70, 1), (128, 1), (33, 1), (100, 1)]
    c = _padded(_paged_case(rng, BF16, 8, 64, 8, 16, seqs), seqs, 4, 2 ** 20 + 3)
    out, lse = _paged_run(c, out=torch.full_like(c["q"], 7.0))
    _paged_check(c, seqs, 8 ** -0.5, out, lse)
    assert (out[4:] == 7).all()


def _sample(rng, heads):
    return np.sort(np.append(rng.choice(heads, 5, replace=False), [0, heads - 1]))


def test_gradients_of_many_column_blocks():
    """257 blocks of 16 columns and 65536 key heads."""
    api = _api()
    rng = np.random.default_rng(63)
    heads, nk, d = 65536, 4100, 8
    rows = [np.sort(rng.permutation(nk)[:30]) for _ in range(5)]
    q, dout = _rand(rng, (5, heads, d), BF16), _rand(rng, (5, heads, d), BF16)
    k = _rand(rng, (nk, 1, d), BF16).expand(-1, heads, -1)
    v = _rand(rng, (nk, 1, d), BF16).expand(-1, heads, -1)
    with api.AttentionPlan(ref.csr(rows, nk), backward=True) as plan:
        out, lse = plan.forward(q, k, v)
        dq, dk, dv = plan.backward(dout, q, k, v, out, lse)
    at = _sample(rng, heads)
    pick = lambda x: ref.f64(x[:, torch.from_numpy(at).cuda()])  # noqa: E731
    want, err = ref.backward(pick(q), pick(k), pick(v), pick(out), ref.f64(lse[:, at]), pick(dout), rows,
                             d ** -0.5, BF16)
    for name, x, w, e in zip(("dq", "dk", "dv"), (dq, dk, dv), want, err):
        ref.check(x[:, torch.from_numpy(at).cuda()], w, e, name)
    named = torch.zeros(nk, dtype=torch.bool)
    named[np.unique(np.concatenate(rows))] = True
    assert not dk[~named].any() and not dv[~named].any()
    assert dv[named].view(-1, heads, d).any(2).all()


def test_joins_of_many_rows_and_heads():
    """1100 of 4400 rows cut into two pieces, 65536 heads: 2^26 results to join and more, of the
    forward pass and of dq; and columns that are cut."""
    api = _api()
    rng = np.random.default_rng(64)
    heads, nk, d = 65536, 100, 8
    rows = [rng.permutation(nk) if i % 4 == 1 else np.zeros(0, int) for i in range(4400)]
    q, k, v = (_rand(rng, (n, 1, d), BF16).expand(-1, heads, -1) for n in (len(rows), nk, nk))
    dout = _rand(rng, (1, heads, d), BF16).expand(len(rows), -1, -1)
    with api.AttentionPlan(ref.csr(rows, nk), backward=True) as plan:
        out, lse = plan.forward(q, k, v)
        dq, dk, dv = plan.backward(dout, q, k, v, out, lse)
    at = _sample(rng, heads)
    some = torch.from_numpy(at).cuda()
    pick = lambda x: ref.f64(x[:, some])  # noqa: E731
    o, l, oe, le = ref.forward(pick(q), pick(k), pick(v), rows, d ** -0.5, BF16)
    ref.check(out[:, some], o, oe, "out")
    ref.check(lse[:, some], l, le, "lse")
    want, err = ref.backward(pick(q), pick(k), pick(v), pick(out), ref.f64(lse[:, some]), pick(dout), rows,
                             d ** -0.5, BF16)
    for name, x, w, e in zip(("dq", "dk", "dv"), (dq, dk, dv), want, err):
        ref.check(x[:, some], w, e, name)
    # every head has the same queries, keys and values
    assert (out == out[:, :1]).all() and (lse == lse[:, :1]).all()
