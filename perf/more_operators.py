"""The cases that the quantised and the latent caches are measured on.

Five operators, each with a plain form (``own`` false) and the library's calls (``own`` true). All
work on paged caches: row s of a CSR matrix lists sequence s's pages, the last tokens of a sequence
are its new ones.

store     new tokens' keys and values quantised into a cache of blocks of 32 values with a power of
          two as scale and 8-bit (e4m3) or 4-bit (e2m1) floating codes, and read back
load      a cache's texts read back
quantized attention of new tokens over such a cache
latent    attention over a cache of one latent vector a token that all heads share (absorbed form:
          queries in the latents' space, values are the vector's first part)
expanded  the same attention with every head's keys and values made from the latents by weights
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BLOCK = 32
# largest code, its exponent, that of the smallest normal code, bits of the fraction
_FORMATS = {"e4m3": (448.0, 8, -6, 3), "e2m1": (6.0, 2, 0, 1)}
_LEAST = -117  # smallest exponent of a scale


def listed():
    return [
        # one user's next token goes into the cache: the smallest call, where the launch counts
        {"name": "store_one", "op": "store", "dtype": "bf16", "format": "e4m3", "seqs": 1, "max_len": 1000, "max_new": 1,
         "page": 16, "pad": 0, "hkv": 8, "d": 128},
        # chunks of sixteen prompts in half precision into 4 bits, in a padded batch
        {"name": "store_prompts", "op": "store", "dtype": "f16", "format": "e2m1", "seqs": 16, "max_len": 4096, "max_new": 2048,
         "page": 64, "pad": 7, "hkv": 8, "d": 128},
        # a whole cache back in bf16, as when texts move to another server
        {"name": "load_texts", "op": "load", "dtype": "bf16", "format": "e4m3", "seqs": 16, "max_len": 16384, "max_new": 16384,
         "page": 16, "pad": 0, "hkv": 8, "d": 128},
        # a few texts in single precision for a look at the numerics: odd pages, 96 values a head
        {"name": "load_odd_f32", "op": "load", "dtype": "f32", "format": "e2m1", "seqs": 3, "max_len": 1777, "max_new": 700,
         "page": 7, "pad": 2, "hkv": 3, "d": 96},
        # one user's next token over 1000
        {"name": "quantized_decode_one", "op": "quantized", "dtype": "bf16", "format": "e4m3", "seqs": 1, "max_len": 1000,
         "max_new": 1, "page": 16, "pad": 0, "hq": 32, "hkv": 8, "d": 128},
        # the next token of 64 users with texts of up to 16K tokens
        {"name": "quantized_decode_batch", "op": "quantized", "dtype": "bf16", "format": "e4m3", "seqs": 64, "max_len": 16384,
         "max_new": 1, "page": 16, "pad": 8, "hq": 64, "hkv": 8, "d": 128},
        # the same in 4 bits and half precision, four guessed tokens for every user
        {"name": "quantized_guess_4bit", "op": "quantized", "dtype": "f16", "format": "e2m1", "seqs": 64, "max_len": 16384,
         "max_new": 4, "page": 32, "pad": 0, "hq": 32, "hkv": 8, "d": 128},
        # chunks of two long prompts over what is cached
        {"name": "quantized_prefill", "op": "quantized", "dtype": "bf16", "format": "e4m3", "seqs": 2, "max_len": 32768,
         "max_new": 2048, "page": 64, "pad": 0, "hq": 32, "hkv": 8, "d": 128},
        # the next token of 32 users with 128 heads over latents of 512 + 64 values
        {"name": "latent_decode_batch", "op": "latent", "dtype": "bf16", "seqs": 32, "max_len": 16384, "max_new": 1, "page": 64,
         "pad": 0, "heads": 128, "dl": 512, "dr": 64},
        # a few tokens of a few users, 20 heads, smaller latents and an odd page
        {"name": "latent_few_f16", "op": "latent", "dtype": "f16", "seqs": 5, "max_len": 3000, "max_new": 3, "page": 24,
         "pad": 3, "heads": 20, "dl": 256, "dr": 32},
        # chunks of two long prompts, 32 heads
        {"name": "expanded_prefill", "op": "expanded", "dtype": "bf16", "seqs": 2, "max_len": 16384, "max_new": 2048, "page": 64,
         "pad": 0, "heads": 32, "dl": 512, "dr": 64, "dn": 128, "dv": 128},
        # short prompts of several users, narrow heads
        {"name": "expanded_short_f16", "op": "expanded", "dtype": "f16", "seqs": 6, "max_len": 700, "max_new": 500, "page": 16,
         "pad": 5, "heads": 9, "dl": 256, "dr": 32, "dn": 64, "dv": 64},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


# bounds of a drawn case: those of the largest listed ones
_MOST = {"store": (1.5e8, 0), "load": (9.0e8, 0), "quantized": (1.1e9, 1.0e12), "latent": (3.2e8, 1.5e11),
         "expanded": (3.2e8, 6.0e11)}


def draw(rng):
    op = rng.choice(("store", "load", "quantized", "quantized", "latent", "latent", "expanded"))
    case = {"op": op, "dtype": rng.choice(("bf16", "bf16", "f16")), "seqs": _spread(rng, 1, 64), "max_len": _spread(rng, 2, 32768),
            "page": rng.choice((1, 7, 16, 24, 32, 64, 128)), "pad": rng.choice((0, 0, 3))}
    if op in ("store", "load", "quantized"):
        case |= {"format": rng.choice(("e4m3", "e2m1")), "hkv": rng.choice((1, 2, 3, 4, 8)), "d": rng.choice((32, 64, 96, 128, 128, 192, 256))}
        if rng.random() < 0.25:
            case["dtype"] = "f32"
        if op == "quantized":
            case["hq"] = case["hkv"] * rng.choice((1, 1, 2, 4, 5, 7, 8))
    elif op == "latent":
        case |= {"heads": _spread(rng, 1, 128), "dl": rng.choice((128, 192, 256, 512, 512)), "dr": rng.choice((32, 64, 64))}
    else:
        case |= {"heads": _spread(rng, 1, 64), "dl": rng.choice((128, 256, 512)), "dr": rng.choice((32, 64, 64)),
                 "dn": rng.choice((64, 128, 128)), "dv": rng.choice((64, 128, 128))}
    if op == "expanded":
        case["max_new"] = _spread(rng, 2, 2048)
    elif op == "load":
        case["max_new"] = case["max_len"]
    else:
        case["max_new"] = 1 if rng.random() < 0.5 else _spread(rng, 2, 2048)
    case["max_new"] = min(case["max_new"], case["max_len"])
    moved, computed = _MOST[op]

    def fits():
        w = work(case)
        heads = case.get("hq", case.get("heads", 0))
        return (w["bytes"] <= moved and (not computed or w["flops"] <= computed)
                and case["seqs"] * case["max_len"] * max(case["max_new"] * heads, 4 * case["hkv"] * case["d"] if op == "quantized" else 0,
                                                         case["dl"] * 4 if op in ("latent", "expanded") else 0,
                                                         heads * 256 if op == "expanded" else 0) <= 2 << 30)

    while case["seqs"] > 1 and not fits():
        case["seqs"] //= 2
    while case["max_len"] > 2 and not fits():
        case["max_len"] //= 2
        case["max_new"] = min(case["max_new"], case["max_len"])
    return case


# ---------------------------------------------------------------- sizes
def _lengths(case):
    """(tokens in the cache, new ones among them) of every sequence, spread over (0, max]."""
    s = torch.arange(case["seqs"], dtype=torch.float64)
    length = (case["max_len"] * (1 - (s * 0.6180339887498949) % 1.0 * 0.97)).long().clamp(min=1)
    if case["op"] == "load" and case["max_new"] == case["max_len"]:
        return length, length
    new = (case["max_new"] * (1 - (s * 0.7548776662466927) % 1.0 * 0.97)).long().clamp(min=1)
    return length, torch.minimum(new, length)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    length, new = _lengths(case)
    cached, tokens = int(length.sum()), int(new.sum())
    pairs = int((new * length - new * (new - 1) // 2).sum())
    if case["op"] in ("latent", "expanded"):
        h, dl, dr = case["heads"], case["dl"], case["dr"]
        moved = size * cached * (dl + dr)
        if case["op"] == "latent":
            return {"bytes": moved + size * tokens * h * (2 * dl + dr) + 4 * tokens * h, "flops": 2 * pairs * h * (2 * dl + dr)}
        dn, dv = case["dn"], case["dv"]
        return {"bytes": moved + size * (h * dl * (dn + dv) + tokens * h * (dn + dr + dv)) + 4 * tokens * h,
                "flops": 2 * cached * dl * h * (dn + dv) + 2 * pairs * h * (dn + dr + dv)}
    d, hkv = case["d"], case["hkv"]
    row = 2 * hkv * (d // (1 if case["format"] == "e4m3" else 2) + d // _BLOCK)  # of the cache: keys and values
    values = 2 * hkv * d * size
    if case["op"] == "store":
        return {"bytes": tokens * (2 * values + row), "flops": 0}
    if case["op"] == "load":
        return {"bytes": tokens * (values + row), "flops": 0}
    return {"bytes": cached * row + tokens * case["hq"] * (2 * d * size + 4), "flops": 4 * pairs * case["hq"] * d}


# ---------------------------------------------------------------- the quantised cache
def _quantize(x, form):
    """(codes, scales) as the cache holds them, of [..., values] floats; 4-bit codes two to a byte,
    the first in the low half."""
    most, high, low, bits = _FORMATS[form]
    x = x.float().unflatten(-1, (-1, _BLOCK))
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, (e - 1 - high + (m > most / 2 ** (high + 1)).int()).clamp(min=_LEAST), _LEAST)
    y = torch.ldexp(x, -e.unsqueeze(-1))
    ex = torch.where(y != 0, torch.frexp(y)[1] - 1, low).clamp(min=low)
    code = (ex - low) * 2 ** bits + torch.round(torch.ldexp(y.abs(), bits - ex)).int()
    sign = torch.signbit(x).int()
    if form == "e4m3":
        return (code + 128 * sign).to(torch.uint8).flatten(-2), (e + 127).to(torch.uint8)
    code = (code + 8 * sign).to(torch.uint8).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (e + 127).to(torch.uint8)


def _code_values(form, device):
    """The value of every code."""
    _, _, low, bits = _FORMATS[form]
    n = 128 if form == "e4m3" else 8
    c = torch.arange(n, device=device)
    ex, f = c >> bits, c & (2 ** bits - 1)
    v = torch.where(ex == 0, torch.ldexp(f.float(), torch.tensor(low - bits, device=device)),
                    torch.ldexp((f + 2 ** bits).float(), ex - 1 + low - bits))
    if form == "e4m3":
        v[127] = math.nan
    return torch.cat((v, -v))


def _dequantize(codes, scales, form):
    """32-bit values of [..., bytes] codes and [..., blocks] scales."""
    table = _code_values(form, codes.device)
    if form == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = table[codes.int()].unflatten(-1, (-1, _BLOCK))
    return torch.ldexp(v, (scales.int() - 127).unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, op, page = _TYPES[case["dtype"]], case["op"], case["page"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    length, new = _lengths(case)
    count = (length + page - 1) // page
    rowptr = torch.zeros(case["seqs"] + 1, dtype=torch.int64)
    rowptr[1:] = torch.cumsum(count, 0)
    pool = int(rowptr[-1]) + 3
    q_rowptr = torch.zeros(case["seqs"] + 1, dtype=torch.int64)
    q_rowptr[1:] = torch.cumsum(new, 0)
    tokens = int(q_rowptr[-1]) + case["pad"]
    order = torch.randperm(pool, generator=gen, device="cuda")[: pool - 3]
    st = {"op": op, "case": case, "pages": order.to(torch.int32), "rowptr": rowptr.cuda(), "q_rowptr": q_rowptr.cuda(),
          "length": length.cuda(), "max_q": int(new.max()), "max_len": int(length.max()), "tokens": tokens, "dtype": dtype, "page": page}
    if op in ("latent", "expanded"):
        h, dl, dr = case["heads"], case["dl"], case["dr"]
        dk = dl + dr if op == "latent" else case["dn"] + dr
        dv = dl if op == "latent" else case["dv"]
        st |= {"q": normal(tokens, h, dk).to(dtype), "cache": normal(pool, page, dl + dr).to(dtype), "dl": dl,
               # queries of absorbed heads have the scale of the heads that they came from
               "scale": (128 + dr) ** -0.5 if op == "latent" else dk ** -0.5,
               "out": torch.zeros(tokens, h, dv, dtype=dtype, device="cuda"), "lse": torch.zeros(tokens, h, device="cuda")}
        if op == "expanded":
            st |= {"w_k": (normal(h, case["dn"], dl) * dl ** -0.5).to(dtype), "w_v": (normal(h, dv, dl) * dl ** -0.5).to(dtype)}
    else:
        form, hkv, d = case["format"], case["hkv"], case["d"]
        st |= {"form": form, "scale": d ** -0.5}
        # some channels of keys are larger than others
        channel = torch.exp(0.5 * normal(hkv, d))
        packed = d if form == "e4m3" else d // 2
        for name in ("k", "v"):
            codes = torch.zeros(pool, page, hkv, packed, dtype=torch.uint8, device="cuda")
            scales = torch.zeros(pool, page, hkv, d // _BLOCK, dtype=torch.uint8, device="cuda")
            if op != "store":
                step = max(1, (1 << 26) // (page * hkv * d))
                for a in range(0, pool, step):
                    x = normal(min(step, pool - a), page, hkv, d)
                    codes[a:a + step], scales[a:a + step] = _quantize(x * channel if name == "k" else x, form)
            st[name + "_codes"], st[name + "_scales"] = codes, scales
        if op == "quantized":
            st |= {"q": normal(tokens, case["hq"], d).to(dtype), "out": torch.zeros(tokens, case["hq"], d, dtype=dtype, device="cuda"),
                   "lse": torch.zeros(tokens, case["hq"], device="cuda")}
        else:
            if op == "store":  # as one projection leaves them
                kv = normal(tokens, 2 * hkv, d)
                kv[:, :hkv] *= channel
                kv = kv.to(dtype)
                st |= {"k": kv[:, :hkv], "v": kv[:, hkv:]}
            st |= {"k_out": torch.zeros(tokens, hkv, d, dtype=dtype, device="cuda"), "v_out": torch.zeros(tokens, hkv, d, dtype=dtype, device="cuda")}
    if own:
        from spgemm_irregular_matrices_amd import binding

        st["table"] = binding.DeviceCSR(case["seqs"], pool, st["rowptr"], st["pages"], None)
        if op in ("latent", "expanded"):
            from spgemm_irregular_matrices_amd import latent

            st["call"] = latent.latent_attention if op == "latent" else latent.latent_attention_expanded
        else:
            from spgemm_irregular_matrices_amd import cache

            st["store"] = cache.QuantizedCache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], form)
    return st


# ---------------------------------------------------------------- plain forms
def _places(st):
    """(rows, their pages, their slots) of the batch's new tokens."""
    first, length = st["q_rowptr"][:-1], st["length"]
    new = st["q_rowptr"][1:] - first
    t = torch.arange(st["max_q"], device=first.device)
    inside = t < new[:, None]
    row = (first[:, None] + t)[inside]
    at = ((length - new)[:, None] + t)[inside]
    seq = torch.arange(first.numel(), device=first.device)[:, None].expand_as(inside)[inside]
    return row, st["pages"].long()[st["rowptr"][seq] + at // st["page"]], at % st["page"]


def _store(st):
    row, page, slot = _places(st)
    for name in ("k", "v"):
        codes, scales = _quantize(st[name][row], st["form"])
        st[name + "_codes"][page, slot] = codes
        st[name + "_scales"][page, slot] = scales
    return _load(st)


def _load(st):
    row, page, slot = _places(st)
    for name in ("k", "v"):
        values = _dequantize(st[name + "_codes"][page, slot], st[name + "_scales"][page, slot], st["form"])
        st[name + "_out"][row] = values.to(st["dtype"])
    return st["k_out"], st["v_out"]


def _attend(st, q, k, v, hkv):
    """Softmax attention of the new tokens: q [tokens, heads, dk], and k(at, slot), v(at, slot) the
    rows [sequences, tokens, kv heads, values] of the cache at these pages and slots."""
    dev = q.device
    first, length = st["q_rowptr"][:-1], st["length"]
    new = st["q_rowptr"][1:] - first
    t, j = torch.arange(st["max_q"], device=dev), torch.arange(st["max_len"], device=dev)
    inside = t < new[:, None]
    where = torch.where(inside, first[:, None] + t, 0)
    q = q.float()[where].unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    there = j < length[:, None]
    at = st["pages"].long()[torch.where(there, st["rowptr"][:-1, None] + j // st["page"], 0)]
    keys = k(at, j % st["page"]).transpose(1, 2)
    s = torch.matmul(q, keys.transpose(2, 3).contiguous()).unflatten(2, (-1, st["max_q"])) * st["scale"]
    del keys
    seen = j <= (length - new)[:, None, None] + t[:, None]
    s = s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    values = (v(at, j % st["page"]) * there[:, :, None, None]).transpose(1, 2).contiguous()
    out = torch.matmul(p.flatten(2, 3), values).unflatten(2, (-1, st["max_q"])) / total
    lse = (top + torch.log(total)).squeeze(-1)
    st["out"][where[inside]] = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[inside].to(st["dtype"])
    st["lse"][where[inside]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[inside]
    return st["out"], st["lse"]


def _quantized(st):
    def values(name):
        return lambda at, slot: _dequantize(st[name + "_codes"][at, slot], st[name + "_scales"][at, slot], st["form"])

    return _attend(st, st["q"], values("k"), values("v"), st["case"]["hkv"])


def _latent(st):
    c, dl = st["cache"], st["dl"]
    return _attend(st, st["q"], lambda at, slot: c[at, slot].float().unsqueeze(2), lambda at, slot: c[at, slot, :dl].float().unsqueeze(2), 1)


def _expanded(st):
    c, dl, h = st["cache"], st["dl"], st["case"]["heads"]

    def made(at, slot, w):
        x = c[at, slot, :dl].float()
        return torch.matmul(x, w.float().flatten(0, 1).T.contiguous()).unflatten(-1, (h, -1))

    def keys(at, slot):
        turned = c[at, slot, dl:].float().unsqueeze(2).expand(-1, -1, h, -1)
        return torch.cat((made(at, slot, st["w_k"]), turned), -1)

    return _attend(st, st["q"], keys, lambda at, slot: made(at, slot, st["w_v"]), h)


def run(st):
    if not own:
        return {"store": _store, "load": _load, "quantized": _quantized, "latent": _latent, "expanded": _expanded}[st["op"]](st)
    batch = {"max_q": st["max_q"], "max_len": st["max_len"]}
    index = st["table"], st["q_rowptr"], st["length"]
    if st["op"] in ("store", "load"):
        if st["op"] == "store":
            st["store"].write(st["k"], st["v"], *index, **batch)
        return st["store"].read(*index, **batch, k=st["k_out"], v=st["v_out"])
    result = {"scale": st["scale"], "out": st["out"], "lse": st["lse"]}
    if st["op"] == "quantized":
        return st["store"].attention(st["q"], *index, **batch, **result)
    if st["op"] == "latent":
        return st["call"](st["q"], st["cache"], *index, **batch, value_dim=st["dl"], **result)
    return st["call"](st["q"], st["cache"], st["w_k"], st["w_v"], *index, **batch, **result)


# ---------------------------------------------------------------- 64 bits
def _nearest(x, form):
    """What a cache keeps of [rows, values] 64-bit numbers: the nearest of all codes, of two equally
    near ones that with the even number."""
    most = _FORMATS[form][0]
    if form == "e4m3":
        table = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    else:
        table = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    table = torch.tensor(table, dtype=torch.float64, device=x.device)
    middle = (table[1:] + table[:-1]) / 2
    x = x.unflatten(-1, (-1, _BLOCK))
    top = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2((top / most).clamp(min=2.0 ** -200))) - 1
    for _ in range(3):
        e = torch.where(top > most * torch.exp2(e), e + 1, e)
    scale = torch.exp2(e.clamp(min=_LEAST))
    y = (x / scale).abs()
    low, high = torch.bucketize(y, middle), torch.bucketize(y, middle, right=True)
    return (torch.sign(x) * table[torch.where(low % 2 == 0, low, high)] * scale).flatten(-2)


def _decode64(codes, scales, form):
    """[rows, bytes] and [rows, blocks] as 64-bit values."""
    c = codes.long()
    if form == "e2m1":
        c = torch.stack((c % 16, c // 16), -1).flatten(-2)
        sign, c = 1 - 2 * (c // 8), c % 8
        v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=c.device)[c]
    else:
        sign, c = 1 - 2 * (c // 128), c % 128
        v = torch.where(c < 8, c * 2.0 ** -9, (8 + c % 8) * torch.exp2((c // 8).double() - 10))
    return sign * v * torch.exp2(scales.double() - 127).repeat_interleave(_BLOCK, -1)


def exact(case, seed):
    """One sequence, and of the attention one head and a block of rows, at a time."""
    st = prepare(case, seed)
    op, page = case["op"], case["page"]
    starts, firsts, lens = st["rowptr"].tolist(), st["q_rowptr"].tolist(), st["length"].tolist()
    if op in ("store", "load"):
        result = []
        for name in ("k", "v"):
            out = torch.zeros(st["tokens"], case["hkv"], case["d"], dtype=torch.float64, device="cuda")
            for s, n in enumerate(lens):
                a, b = firsts[s], firsts[s + 1]
                if op == "store":
                    out[a:b] = _nearest(st[name][a:b].double(), st["form"])
                else:
                    ids = st["pages"][starts[s]:starts[s + 1]].long()
                    c, x = (st[name + part][ids].flatten(0, 1)[n - (b - a):n] for part in ("_codes", "_scales"))
                    out[a:b] = _decode64(c, x, st["form"])
            result.append(out)
        return tuple(result)
    out, lse = st["out"].double(), st["lse"].double()
    heads = out.shape[1]
    for s, n in enumerate(lens):
        ids = st["pages"][starts[s]:starts[s + 1]].long()
        if op == "quantized":
            kv = [_decode64(*(st[name + part][ids].flatten(0, 1)[:n] for part in ("_codes", "_scales")), st["form"]) for name in "kv"]
        else:
            rows = st["cache"][ids].flatten(0, 1)[:n].double()
        for h in range(heads):
            if op == "quantized":
                keys, vals = (x[:, h // (heads // case["hkv"])] for x in kv)
            elif op == "latent":
                keys, vals = rows, rows[:, :case["dl"]]
            else:
                made = rows[:, :case["dl"]]
                keys = torch.cat((made @ st["w_k"][h].double().T, rows[:, case["dl"]:]), 1)
                vals = made @ st["w_v"][h].double().T
            for a in range(firsts[s], firsts[s + 1], 512):
                b = min(a + 512, firsts[s + 1])
                last = n - firsts[s + 1] + torch.arange(a, b, device="cuda")
                x = st["q"][a:b, h].double() @ keys.T * st["scale"]
                x = x.masked_fill(torch.arange(n, device="cuda") > last[:, None], -math.inf)
                lse[a:b, h] = torch.logsumexp(x, -1)
                out[a:b, h] = torch.softmax(x, -1) @ vals
    return out, lse
