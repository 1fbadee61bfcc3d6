"""The quantised cache's C ABI and binding (CPU only): exports, struct layouts,
limits of sizes, and the refusals that need no GPU."""
import ctypes
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

from spgemm_irregular_matrices_amd import attention, binding, cache  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "spgemm_cache.h")
STRUCTS = {"spgemm_mx_bytes": cache.MxBytes, "spgemm_mx_cache": cache.MxCache}
EXPORTS = set(cache.EXPORTS)


def test_library_exports_every_declared_symbol():
    names = re.findall(r"SPGEMM_API\s+[\w\s\*]+?\b(spgemm_\w+)\s*\(", open(HEADER).read())
    assert set(names) == EXPORTS
    lib = cache.load()
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layout_matches_header(tmp_path):
    lines = []
    for name, s in STRUCTS.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f[0]}));' for f in s._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "spgemm_cache.h"\n'
                    "int main(void) {" + "\n".join(lines) + "return 0;}")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(prog),
                           "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    want = []
    for s in STRUCTS.values():
        want.append(ctypes.sizeof(s))
        want += [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want


def _batch(seqs=4, tokens=4, max_new=1, max_length=1000, npages=10):
    table = binding.CSRStruct(seqs, npages, 0, None, None, None)
    return attention.PagedBatch(ctypes.pointer(table), None, None, tokens, max_new, max_length)


def _mx_bytes(desc, **sizes):
    n = ctypes.c_int64(-1)
    batch = _batch(**sizes)
    return cache.load().spgemm_mx_attention_workspace(ctypes.byref(desc), ctypes.byref(batch),
                                                      ctypes.byref(n)), n.value


def test_descriptions_are_checked():
    D = attention.Desc
    for good in (D(0, 8, 2, 128, 0.1), D(1, 8, 2, 32, 0.1), D(2, 7, 7, 96, 0.1), D(0, 8, 1, 256, 0.1)):
        assert _mx_bytes(good)[0] == 0
    for bad in (D(3, 8, 2, 128, 0.1), D(0, 8, 3, 128, 0.1), D(0, 8, 2, 80, 0.1), D(0, 8, 2, 16, 0.1),
                D(0, 8, 2, 0, 0.1), D(0, 8, 2, 288, 0.1), D(0, 8, 2, 128, float("nan"))):
        assert _mx_bytes(bad)[0] == -1


def test_sizes_are_checked():
    d = attention.Desc(0, 8, 2, 128, 0.1)
    for bad in (dict(seqs=-1), dict(tokens=-1), dict(max_new=-1), dict(max_length=-1)):
        assert _mx_bytes(d, **bad)[0] == -1
    for big in (dict(tokens=1 << 29), dict(max_length=1 << 31), dict(seqs=1 << 31), dict(tokens=1 << 61)):
        assert _mx_bytes(d, **big)[0] == -4
    assert _mx_bytes(d, max_length=32) == (0, 0)
    rc, n = _mx_bytes(d, max_length=1000)  # pieces: dim floats and two more per row each
    assert rc == 0 and n > 0
    one = attention.Desc(0, 1, 1, 128, 0.1)
    assert _mx_bytes(one, tokens=2 ** 30, max_new=2 ** 30, max_length=2 ** 30)[0] == 0


def test_null_and_broken_arguments_are_refused():
    """No pointer of these calls is read: each is refused for what it lacks."""
    lib, ref = cache.load(), ctypes.byref
    d = attention.Desc(0, 2, 2, 64, 0.1)
    rows = attention.Rows(1 << 20, 128, 64)
    part = cache.MxBytes(1 << 20, 2048, 128, 64)
    scales = cache.MxBytes(3, 64, 4, 2)
    good = cache.MxCache(0, 0, 10, 16, part, scales, part, scales)
    batch = _batch()
    assert lib.spgemm_mx_write(None, *[None] * 5) == -1
    assert lib.spgemm_mx_read(None, *[None] * 5) == -1
    assert lib.spgemm_mx_attention(ref(d), *[None] * 6, 0, None) == -1
    assert lib.spgemm_mx_attention_workspace(ref(d), ref(batch), None) == -1

    def codes(c=good, k=rows, v=rows, b=batch, desc=d):
        n = ctypes.c_int64(0)
        lib.spgemm_mx_attention_workspace(ref(desc), ref(b), ref(n))
        a = lib.spgemm_mx_write(ref(desc), ref(k), ref(v), ref(c), ref(b), None)
        r = lib.spgemm_mx_read(ref(desc), ref(c), ref(b), ref(k), ref(v), None)
        t = lib.spgemm_mx_attention(ref(desc), ref(k), ref(c), ref(b), ref(v), None, 256, n.value, None)
        assert a == r == t, (a, r, t)
        return a

    assert codes() == -1  # row pointers are missing
    table = binding.CSRStruct(4, 10, 0, 256, None, None)
    whole = attention.PagedBatch(ctypes.pointer(table), 256, 256, 4, 1, 1000)
    for bad in (cache.MxCache(2, 0, 10, 16, part, scales, part, scales),
                cache.MxCache(0, 1, 10, 16, part, scales, part, scales),
                cache.MxCache(0, 0, 10, 0, part, scales, part, scales),
                cache.MxCache(0, 0, 9, 16, part, scales, part, scales),
                cache.MxCache(0, 0, 10, 16, cache.MxBytes(8, 2048, 128, 64), scales, part, scales),
                cache.MxCache(0, 0, 10, 16, cache.MxBytes(None, 2048, 128, 64), scales, part, scales),
                cache.MxCache(0, 0, 10, 16, part, scales, cache.MxBytes(1 << 20, 2048, 120, 64), scales),
                cache.MxCache(0, 0, 10, 16, part, scales, cache.MxBytes(1 << 20, 2048, 128, -64), scales),
                cache.MxCache(0, 0, 10, 16, part, cache.MxBytes(None, 64, 4, 2), part, scales),
                cache.MxCache(0, 0, 10, 16, part, scales, part, cache.MxBytes(3, -64, 4, 2))):
        assert codes(bad, b=whole) == -1
    # pages so far apart that a place in units of 16 bytes passes 32 bits
    far = cache.MxCache(0, 0, 10, 16, cache.MxBytes(1 << 20, (1 << 33) + 16, 128, 64), scales, part, scales)
    assert codes(far, b=whole) == -4
    for bad in (attention.Rows(None, 128, 64), attention.Rows(8, 128, 64), attention.Rows(1 << 20, 124, 64)):
        assert codes(k=bad, b=whole) == -1 and codes(v=bad, b=whole) == -1
    # without work nothing of the cache is used
    none = attention.PagedBatch(ctypes.pointer(table), 256, 256, 0, 1, 1000)
    assert codes(b=none) == 0


def _cache(**changed):
    shape = (3, 16, 2, 64)
    parts = dict(k_codes=torch.zeros(shape, dtype=torch.uint8), v_codes=torch.zeros(shape, dtype=torch.uint8),
                 k_scales=torch.zeros(*shape[:3], 2, dtype=torch.uint8),
                 v_scales=torch.zeros(*shape[:3], 2, dtype=torch.uint8), format="e4m3")
    return cache.QuantizedCache(**{**parts, **changed})


def test_caches_are_checked():
    c = _cache()
    assert (c.npages, c.slots, c.heads, c.dim) == (3, 16, 2, 64)
    assert _cache(format="e2m1", k_scales=torch.zeros(3, 16, 2, 4, dtype=torch.uint8),
                  v_scales=torch.zeros(3, 16, 2, 4, dtype=torch.uint8)).dim == 128
    z = torch.zeros
    for bad in (dict(format="e5m2"), dict(k_codes=z(3, 16, 128, dtype=torch.uint8)),
                dict(k_codes=z(3, 16, 2, 80, dtype=torch.uint8)), dict(v_codes=z(3, 16, 2, 32, dtype=torch.uint8)),
                dict(v_codes=z(3, 16, 2, 64, dtype=torch.int8)), dict(k_scales=z(3, 16, 2, 1, dtype=torch.uint8)),
                dict(v_scales=z(3, 16, 1, 2, dtype=torch.uint8)),
                dict(v_codes=z(3, 16, 64, 2, dtype=torch.uint8).transpose(2, 3))):
        with pytest.raises(ValueError):
            _cache(**bad)
    with pytest.raises(ValueError):
        cache.QuantizedCache.empty(1, 16, 1, 80, device="cpu")
    with pytest.raises(ValueError):
        cache.QuantizedCache.empty(1, 16, 1, 64, "int8", device="cpu")
    e = cache.QuantizedCache.empty(2, 16, 3, 64, "e2m1", device="cpu")
    assert e.k_codes.shape == (2, 16, 3, 32) and e.v_scales.shape == (2, 16, 3, 2)


def test_calls_are_refused_before_any_work():
    """Shapes, gradients, and tensors that are not on a GPU."""
    c = _cache()
    table = binding.DeviceCSR(1, 3, torch.tensor([0, 1]), torch.zeros(1, dtype=torch.int32), None)
    index = (table, torch.tensor([0, 1]), torch.tensor([1]), 1, 1)
    row, q = torch.zeros(1, 2, 64), torch.zeros(1, 4, 64)
    for k, v in ((torch.zeros(1, 2, 32), row), (row, torch.zeros(2, 2, 64)), (row.long(), row.long()),
                 (row, row.half())):
        with pytest.raises(ValueError):
            c.write(k, v, *index)
    with pytest.raises(ValueError):
        c.attention(torch.zeros(1, 4, 32), *index)
    for x, y in ((True, False), (False, True)):
        k, v = row.clone().requires_grad_(x), row.clone().requires_grad_(y)
        with pytest.raises(ValueError, match="autograd"):
            c.write(k, v, *index)
        with pytest.raises(ValueError, match="autograd"):
            c.read(*index, k=k, v=v)
    with pytest.raises(ValueError, match="autograd"):
        c.attention(q.clone().requires_grad_(True), *index)
    for call in (lambda: c.write(row, row, *index), lambda: c.read(*index, tokens=1),
                 lambda: c.attention(q, *index)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
