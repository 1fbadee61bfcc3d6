"""The attention entry points' C ABI (CPU only): exports, struct layouts, and
the refusals that need no GPU."""
import ctypes
import os
import re
import subprocess

import pytest

from spgemm_irregular_matrices_amd import attention, binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "spgemm_attention.h")


def test_library_exports_every_declared_symbol():
    names = re.findall(r"SPGEMM_API\s+[\w\s\*]+?\b(spgemm_\w+)\s*\(", open(HEADER).read())
    assert set(names) == set(attention.EXPORTS)
    lib = attention.load()
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layout_matches_header(tmp_path):
    structs = {"spgemm_attention_desc": attention.Desc, "spgemm_rows": attention.Rows,
               "spgemm_paged_cache": attention.PagedCache, "spgemm_paged_batch": attention.PagedBatch}
    lines = []
    for name, s in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f[0]}));' for f in s._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "spgemm_attention.h"\n'
                    "int main(void) {" + "\n".join(lines) + "return 0;}")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(prog),
                           "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    want = []
    for s in structs.values():
        want.append(ctypes.sizeof(s))
        want += [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want


def _paged_bytes(desc, seqs=4, tokens=4, max_new=1, max_length=1000):
    lib = attention.load()
    table = binding.CSRStruct(seqs, 10, 0, None, None, None)
    batch = attention.PagedBatch(ctypes.pointer(table), None, None, tokens, max_new, max_length)
    n = ctypes.c_int64(-1)
    rc = lib.spgemm_paged_attention_workspace(ctypes.byref(desc), ctypes.byref(batch), ctypes.byref(n))
    return rc, n.value


def test_descriptions_are_checked():
    D = attention.Desc
    assert _paged_bytes(D(0, 8, 2, 128, 0.1))[0] == 0
    for bad in (D(3, 8, 2, 128, 0.1), D(-1, 8, 2, 128, 0.1), D(0, 8, 3, 128, 0.1), D(0, 0, 1, 128, 0.1),
                D(0, 8, 0, 128, 0.1), D(0, 8, -2, 128, 0.1), D(0, 8, 2, 0, 0.1), D(0, 8, 2, 12, 0.1),
                D(2, 8, 2, 6, 0.1), D(0, 8, 2, 264, 0.1), D(0, 8, 2, 128, float("nan")),
                D(0, 8, 2, 128, float("inf")), D(0, 1 << 17, 1, 128, 0.1)):
        assert _paged_bytes(bad)[0] == -1
    assert _paged_bytes(D(2, 8, 2, 4, 0.1))[0] == 0


def test_paged_sizes_are_checked():
    d = attention.Desc(0, 8, 2, 128, 0.1)
    for bad in (dict(seqs=-1), dict(tokens=-1), dict(max_new=-1), dict(max_length=-1)):
        assert _paged_bytes(d, **bad)[0] == -1
    for big in (dict(tokens=1 << 29), dict(max_length=1 << 31), dict(seqs=1 << 31)):
        assert _paged_bytes(d, **big)[0] == -4
    assert _paged_bytes(d, max_length=32) == (0, 0)
    rc, n = _paged_bytes(d, max_length=1000)  # pieces: dim floats and two more per row each
    assert rc == 0 and n > 0
    assert _paged_bytes(d, seqs=0, tokens=0)[0] == 0


def test_null_arguments_are_refused():
    lib = attention.load()
    d = attention.Desc(0, 8, 2, 128, 0.1)
    n = ctypes.c_int64()
    assert lib.spgemm_attention_plan_create(None, None, 0, None) == -1
    h = ctypes.c_void_p()
    assert lib.spgemm_attention_plan_create(ctypes.byref(h), None, 0, None) == -1 and not h.value
    assert lib.spgemm_attention_workspace(None, ctypes.byref(d), 0, ctypes.byref(n)) == -1
    assert lib.spgemm_attention_forward(None, ctypes.byref(d), *[None] * 6, 0, None) == -1
    assert lib.spgemm_attention_backward(None, ctypes.byref(d), *[None] * 10, 0, None) == -1
    assert lib.spgemm_paged_attention(ctypes.byref(d), *[None] * 6, 0, None) == -1
    lib.spgemm_attention_plan_destroy(None)


def test_no_gpu_call_fails_loudly():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("GPU present")
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    mask = binding.DeviceCSR(1, 1, torch.tensor([0, 1]), torch.zeros(1, dtype=torch.int32), None)
    with pytest.raises(ValueError):
        attention.AttentionPlan(mask)
    cache = torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attention.paged_attention(q, cache, cache, mask, torch.tensor([0, 1]), torch.tensor([1]), 1, 1)


def test_paged_sizes_at_their_limits():
    """A tile of up to 128 rows begins inside the last sequence's rows, so its end fits 32 bits
    only up to 2^31 - 128 pairs of token and query head; larger products must not wrap around."""
    d = attention.Desc(0, 8, 8, 128, 0.1)
    most = (2 ** 31 - 128) // 8
    assert _paged_bytes(d, tokens=most, max_length=32) == (0, 0)
    for tokens in (most + 1, 2 ** 28, 2 ** 61, 2 ** 61 + 1, 2 ** 63 - 1):
        assert _paged_bytes(d, tokens=tokens, max_length=32)[0] == -4, tokens
    many = attention.Desc(0, 65536, 1, 128, 0.1)
    for tokens in (2 ** 15, 2 ** 47, 2 ** 48, 2 ** 48 + 1):
        assert _paged_bytes(many, tokens=tokens, max_length=32)[0] == -4, tokens
    one = attention.Desc(0, 1, 1, 128, 0.1)
    assert _paged_bytes(one, tokens=2 ** 30, max_new=2 ** 30, max_length=2 ** 30)[0] == 0
    for tokens in (2 ** 30 + 1, 2 ** 62):
        assert _paged_bytes(one, tokens=tokens, max_length=32)[0] == -4, tokens
