"""Quantised caches and attention over a cache, in 64 bits on the host, straight
from their definitions, with a bound on the error of each result.

The bounds count roundings as ``attention_ref`` does (u: half a step of the
tensors' type, e = 2^-24 that of a float), with two more numbers per call:
  terms    products and sums of one score, in floats
  weight   relative rounding of a weight before the second product
"""
import numpy as np
import torch

from tests import attention_ref as ref

E, U = ref.E, ref.U
BLOCK = 32
# (largest code, exponent of its power of two, smallest normal exponent, bits of fraction)
FORMATS = {"e4m3": (448.0, 8, -6, 3), "e2m1": (6.0, 2, 0, 1)}
# Bfloat16 parts of a query and of a weight; what a weight loses: its own rounding
# to 8 bits; cut to 8 bits (less than 2^-7 of it is left), the rest rounded to 8;
# nothing.
PARTS = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}
WEIGHT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -15, torch.float32: 0.0}


def code_table(form):
    """The value of every code, by its number."""
    if form == "e4m3":
        table = [m * 2.0 ** -9 for m in range(8)]
        table += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
        table[127] = np.nan
    else:
        table = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return np.array(table + [-x for x in table])


def quantize(x, form):
    """(codes, scale bytes) of [..., dim] 64-bit values; one code to a number."""
    most = FORMATS[form][0]
    table = code_table(form)
    half = len(table) // 2
    known = table[:half][np.isfinite(table[:half])]
    x = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    top = np.abs(x).max(-1)
    wild = ~np.isfinite(x).all(-1)
    e = np.full(top.shape, -117)
    while (past := ~wild & (top > most * np.exp2(e.astype(float)))).any():
        e[past] += 1
    with np.errstate(invalid="ignore"):
        y = np.abs(np.where(wild[..., None], 0.0, x)) / np.exp2(e.astype(float))[..., None]
    middle = (known[1:] + known[:-1]) / 2
    low, high = np.searchsorted(middle, y, side="left"), np.searchsorted(middle, y, side="right")
    codes = np.where(low % 2 == 0, low, high) + half * np.signbit(x)
    return codes.reshape(*x.shape[:-2], x.shape[-2] * BLOCK), np.where(wild, 255, e + 127)


def values(codes, scales, form):
    """What numbers of codes and scale bytes stand for."""
    with np.errstate(over="ignore"):
        s = np.where(scales == 255, np.nan, np.exp2(scales.astype(float) - 127))
    return (code_table(form)[codes].reshape(*scales.shape, BLOCK) * s[..., None]).reshape(codes.shape)


def unpack(codes, form):
    """Numbers of the codes of a cache's bytes."""
    codes = codes.astype(np.int64)
    if form == "e4m3":
        return codes
    return np.stack((codes % 16, codes // 16), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def pack(codes, form):
    """Bytes of a cache from its codes' numbers."""
    return (codes if form == "e4m3" else codes[..., 0::2] + 16 * codes[..., 1::2]).astype(np.uint8)


def attend(q, k, v, first, scale, dtype, terms, weight, parts=1, key_error=0.0, value_error=0.0):
    """New tokens first, first + 1, ... of one sequence: q [m, H, dk], k [n, HK,
    dk], v [n, HK, dv]; token t sees keys 0 to first + t. Returns out, lse and
    their error bounds. key_error, value_error: relative error of each key and
    value that enters, against the magnitudes that made it (k_mag, v_mag)."""
    m, H, _ = q.shape
    n, HK, dv = v.shape
    u = U[dtype]
    out, out_err = np.zeros((m, H, dv)), np.zeros((m, H, dv))
    lse, lse_err = np.full((m, H), -np.inf), np.zeros((m, H))
    seen = np.arange(n) <= first + np.arange(m)[:, None]
    ke, ve = key_error, value_error
    for h in range(H):
        g = h // (H // HK)
        kk, vv = k[:, g], v[:, g]
        s = np.where(seen, scale * (q[:, h] @ kk.T), -np.inf)
        mag = abs(scale) * (np.abs(q[:, h]) @ np.abs(kk).T)
        es = (terms + 4) * E * mag + 4 * E * np.where(seen, np.abs(s), 0)
        if np.ndim(ke):
            es = es + abs(scale) * (np.abs(q[:, h]) @ ke[:, g].T)
        top = s.max(-1, keepdims=True)
        es = np.where(seen, es + 4 * E * np.abs(top) + 4 * E, 0)
        w = np.exp(s - top)
        l = w.sum(-1, keepdims=True)
        p = w / l
        count = seen.sum(-1, keepdims=True)
        lse[:, h] = (top + np.log(l))[:, 0]
        worst = es.max(-1, keepdims=True)
        lse_err[:, h] = (2 * worst + count * E + 8 * E * (1 + np.abs(lse[:, h])[:, None] + np.abs(top)))[:, 0]
        out[:, h] = p @ vv
        per = es + worst + weight + (2 * parts * count + 16) * E
        out_err[:, h] = u * np.abs(out[:, h]) + 1.01 * ((p * per) @ np.abs(vv))
        if np.ndim(ve):
            out_err[:, h] += 1.01 * (p @ ve[:, g])
        if dtype == torch.float16:  # a result below its normal range
            out_err[:, h] += 2.0 ** -25
    return out, lse, out_err, lse_err
