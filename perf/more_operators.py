"""Microscaled operators, as they are measured: quantisation of matrices to 4- and 8-bit
floating point with a power-of-two scale per 32 values, the linear layer over such matrices
and its gradients, a paged cache of keys and values that is quantised as it is written, and
attention of new tokens over that cache.

A group of 32 consecutive values of a row holds codes of E2M1 ("fp4": 0, 1/2, 1, 3/2, 2, 3, 4, 6
and their negatives, two to a byte, the even column in the low four bits) or E4M3 ("fp8", up
to 448), and one scale byte e for 2^(e - 127).
"""
import math

import torch

own = False  # False: plain torch forms; True: the framework's operators

GROUP = 32  # values that share one scale
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FORMATS = ("fp4", "fp8")
TOP = {"fp4": 2, "fp8": 8}  # exponent of the format's largest power of two
LIMIT = {"fp4": 6.0, "fp8": 448.0}

LARGEST = 8192 * 4096 * 14336  # B M N of the largest product listed
LONGEST = 16 * 2048 * 16384 * 128  # new tokens x keys x width of the largest attention drawn


def _quantise(name, rows, cols, dtype, fmt):
    return {"name": name, "op": "quantise", "rows": rows, "cols": cols, "dtype": dtype,
            "fmt": fmt}


def _linear(name, B, M, N, dtype, fmt, bias=False, residual=False):
    return {"name": name, "op": "linear", "B": B, "M": M, "N": N, "dtype": dtype, "fmt": fmt,
            "bias": bias, "residual": residual}


def _backward(name, B, M, N, dtype, fmt, dw=True):
    return {"name": name, "op": "backward", "B": B, "M": M, "N": N, "dtype": dtype, "fmt": fmt,
            "dw": dw}


def _cached(name, op, seqs, new, length, heads, group, dim, page, dtype, fmt):
    """seqs sequences of length[0] .. length[1] tokens, new[0] .. new[1] of them new; heads
    of keys and values, each shared by group heads of queries."""
    return {"name": name, "op": op, "seqs": seqs, "new_lo": new[0], "new_hi": new[1],
            "len_lo": length[0], "len_hi": length[1], "heads": heads, "group": group,
            "dim": dim, "page": page, "dtype": dtype, "fmt": fmt}


def listed():
    return [
        # a 1B-class projection's weights quantised to four bits, and read back
        _quantise("weights-fp4-2048", 2048, 2048, "f32", "fp4"),
        # a long sequence's MLP activations kept in eight bits
        _quantise("activations-fp8-16384x14336", 16384, 14336, "bf16", "fp8"),
        # one token through an 8B-class up projection: latency, and the weights' bytes
        _linear("token-fp8-14336x4096", 1, 14336, 4096, "bf16", "fp8"),
        # drafted or ragged tokens of some sequences, both sides in four bits, with bias
        _linear("tokens100-fp4-4096", 100, 4096, 4096, "f16", "fp4", bias=True),
        # a long prompt through the down projection: the largest product
        _linear("prompt-fp4-down", 8192, 4096, 14336, "bf16", "fp4", residual=True),
        # fine-tuning steps: gradients of input, matrix and bias from the quantised input
        _backward("grad-fp4-509x2048", 509, 2048, 2048, "bf16", "fp4"),
        _backward("grad-fp8-4096", 4096, 4096, 4096, "f16", "fp8"),
        # one new token of each of 64 sequences put into the cache, and read back
        _cached("append-64", "cache", 64, (1, 1), (500, 8000), 8, 4, 128, 64, "bf16", "fp8"),
        # four prompts put into a 4-bit cache
        _cached("store-prompts-fp4", "cache", 4, (1000, 8192), (1000, 8192), 8, 4, 128, 16,
                "bf16", "fp4"),
        # the next token of a single sequence, 1B-class heads: latency
        _cached("attend-token", "attention", 1, (1, 1), (4001, 4001), 8, 4, 64, 64, "bf16",
                "fp8"),
        # one token of each of 64 sequences: the cache's bytes
        _cached("attend-64-tokens", "attention", 64, (1, 1), (1000, 16000), 8, 4, 128, 64,
                "bf16", "fp8"),
        # chunks of four prompts over what the cache holds of them already
        _cached("attend-chunks", "attention", 4, (511, 2048), (4000, 16384), 8, 4, 128, 32,
                "bf16", "fp8"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantise", "linear", "linear", "backward", "cache", "attention",
                     "attention"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    fmt = rng.choice(FORMATS)
    if op == "quantise":
        case = _quantise("", _log_int(rng, 1, 16384), _log_int(rng, 33, 14336), dtype, fmt)
    elif op in ("linear", "backward"):
        M, N = _log_int(rng, 64, 14336), _log_int(rng, 64, 14336)
        products = 1 if op == "linear" else 2
        B = _log_int(rng, 1, min(16384, max(1, LARGEST // (products * M * N))))
        if op == "linear":
            case = _linear("", B, M, N, dtype, fmt, rng.random() < 0.5, rng.random() < 0.5)
        else:
            case = _backward("", B, M, N, dtype, fmt, rng.random() < 0.7)
    else:
        heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 5, 8))
        dim, page = rng.choice((64, 128, 128, 256)), rng.choice((16, 32, 64, 128))
        seqs = _log_int(rng, 1, 64)
        width = heads * group * dim
        if rng.random() < 0.5:  # single tokens, or a few drafted ones
            new = (1, rng.choice((1, 1, 4)))
            hi = _log_int(rng, 64, 16384)
        else:
            hi = _log_int(rng, 64, 16384)
            most = max(2, LONGEST // (seqs * hi * width))
            new = (1, _log_int(rng, 2, max(2, min(hi, most, 65536 // seqs))))
        case = _cached("", op, seqs, new, (max(new[1], hi // 8), max(new[1], hi)), heads, group,
                       dim, page, dtype, fmt)
    del case["name"]
    return case


def _lengths(case):
    """(new, length) of each sequence, spread evenly over the case's ranges."""
    def spread(lo, hi, s, step):
        return lo + int((s * step) % 1.0 * (hi - lo + 1)) if s else hi

    new = [spread(case["new_lo"], case["new_hi"], s, 0.6180339887) for s in range(case["seqs"])]
    return [(n, max(n, spread(case["len_lo"], case["len_hi"], s, 0.4142135624)))
            for s, n in enumerate(new)]


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _power_of_two(e):
    """2^e exactly, float64, for integers |e| < 1000."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _encode(x, fmt):
    """Plain form of the quantisation along the last dimension, a multiple of 32:
    (one code per value uint8, scale bytes)."""
    v = x.unflatten(-1, (-1, GROUP)).double()
    top = v.abs().amax(-1)
    field = (top.float().view(torch.int32) >> 23) & 255
    e = (field - TOP[fmt]).clamp_min(0)
    e = torch.where(field == 255, field, e)
    q = v * _power_of_two(127 - e).unsqueeze(-1)
    q = torch.where((e == 255).unsqueeze(-1), torch.zeros_like(q), q)
    q = q.clamp(-LIMIT[fmt], LIMIT[fmt]).float()
    if fmt == "fp8":
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        m = q.abs()
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
        m = torch.round(m / step) * step
        code = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4))
        codes = code.to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    return codes.flatten(-2), e.to(torch.uint8)


def _store(codes, fmt):
    """The bytes of codes: two 4-bit codes to a byte."""
    if fmt == "fp8":
        return codes
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _load(stored, fmt):
    if fmt == "fp8":
        return stored
    return torch.stack([stored & 15, stored >> 4], -1).flatten(-2)


def _decode(codes, scale, fmt):
    """Plain form: the float32 values that codes and scale bytes stand for."""
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        m = (codes & 7).float()
        m = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
        v = torch.where(codes >= 8, -m, m)
    e = scale.int().unsqueeze(-1)
    p = _power_of_two(e - 127)
    p = torch.where(e == 255, torch.full_like(p, math.nan), p)
    return (v.unflatten(-1, (-1, GROUP)) * p).float().flatten(-2)


def _whole(x):
    """x with zeros behind its last column up to a whole group."""
    return torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % GROUP))


def _packed(x, fmt):
    """(stored codes, scale bytes) of a matrix."""
    codes, scale = _encode(_whole(x), fmt)
    return _store(codes, fmt).contiguous(), scale.contiguous()


def _values(packed, cols, fmt):
    return _decode(_load(packed[0], fmt), packed[1], fmt)[:, :cols]


def _prepare_cache(case, g, st):
    S, P, H, D = case["seqs"], case["page"], case["heads"], case["dim"]
    fmt, dt = case["fmt"], TYPES[case["dtype"]]
    sizes = _lengths(case)
    pages = [-(-length // P) for _, length in sizes]
    total = sum(pages) + 3  # some pages belong to nobody here
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    st["table"] = torch.full((S, max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(pages):
        st["table"][s, :n] = order[at:at + n]
        at += n
    new = [n for n, _ in sizes]
    st["starts"] = torch.tensor([sum(new[:s]) for s in range(S + 1)], dtype=torch.int32,
                                device="cuda")
    st["lens"] = torch.tensor([length for _, length in sizes], dtype=torch.int32, device="cuda")
    st["sizes"], T = sizes, sum(new)
    if case["op"] == "cache":
        width = D if fmt == "fp8" else D // 2
        st["cache"] = [torch.zeros(total, H, P, w, dtype=torch.uint8, device="cuda")
                       for w in (width, D // GROUP, width, D // GROUP)]
        channel = torch.exp(0.5 * _randn(g, H, D))
        st["k"] = (_randn(g, T, H, D) * channel).to(dt)
        st["v"] = _randn(g, T, H, D).to(dt)
        return
    # keys have channels of different sizes, queries such that scores are of order one
    channel = torch.exp(0.5 * _randn(g, H, 1, D))
    st["cache"] = []
    for what in (channel, None):
        stored, scales = [], []
        for first in range(0, total, 4096):
            x = _randn(g, min(4096, total - first), H, P, D)
            codes, scale = _encode(x if what is None else x * what, fmt)
            stored.append(_store(codes, fmt))
            scales.append(scale)
        st["cache"] += [torch.cat(stored), torch.cat(scales)]
    size = channel.square().mean(-1, keepdim=True).sqrt()
    q = _randn(g, T, H, case["group"], D) / size.view(1, H, 1, 1)
    st["q"] = q.view(T, -1, D).to(dt)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, fmt = TYPES[case["dtype"]], case["fmt"]
    st = {"case": case}
    if case["op"] == "quantise":
        rows, cols = case["rows"], case["cols"]
        if case["dtype"] == "f32":  # weights, rows of different sizes
            st["x"] = _randn(g, rows, cols) * torch.exp(0.3 * _randn(g, rows, 1)) * 0.02
        else:  # activations: a few channels far larger than the others
            st["x"] = (_randn(g, rows, cols) * torch.exp(_randn(g, 1, cols))).to(dt)
        return st
    if case["op"] in ("cache", "attention"):
        _prepare_cache(case, g, st)
        return st
    B, M, N = case["B"], case["M"], case["N"]
    st["w"] = _packed(_randn(g, M, N) * torch.exp(0.3 * _randn(g, M, 1)) / math.sqrt(N), "fp4")
    if case["op"] == "linear":
        st["x"] = (_randn(g, B, N) * torch.exp(0.5 * _randn(g, 1, N))).to(dt)
        st["bias"] = _randn(g, M) if case["bias"] else None
        st["residual"] = _randn(g, B, M).to(dt) if case["residual"] else None
    else:
        st["dy"] = _randn(g, B, M).to(dt)
        st["x"] = _packed(_randn(g, B, N).to(dt), fmt) if case["dw"] else None
    return st


def _run_own(st):
    from trellis_coded_bit_amd import api
    case = st["case"]
    op, fmt = case["op"], case["fmt"]
    if op == "quantise":
        packed = api.mx_pack(st["x"], fmt)
        return {"x": api.mx_unpack(packed, st["x"].dtype), "scale": packed.scale}
    if op in ("linear", "backward"):
        w = api.MxPacked(*st["w"], case["N"], "fp4")
        if op == "linear":
            return {"y": api.mx_linear(st["x"], w, bias=st["bias"], residual=st["residual"],
                                       x_format=fmt)}
        x = None if st["x"] is None else api.MxPacked(*st["x"], case["N"], fmt)
        dx, dw, dbias = api.mx_linear_backward(st["dy"], w, x)
        return {"dx": dx, "dw": dw, "dbias": dbias}
    cache = api.Cache(*st["cache"], fmt)
    where = (st["table"], st["lens"], st["starts"])
    if op == "cache":
        api.cache_write(cache, st["k"], st["v"], *where)
        k, v = api.cache_read(cache, *where, st["k"].shape[0], st["k"].dtype)
        return {"k": k, "v": v}
    return {"o": api.cache_attention(st["q"], cache, *where)}


def _slots(st):
    """Page and place in it of every new token."""
    P, pages, places = st["case"]["page"], [], []
    for s, (n, length) in enumerate(st["sizes"]):
        t = torch.arange(length - n, length, device="cuda")
        pages.append(st["table"][s].long()[t // P])
        places.append(t % P)
    return torch.cat(pages), torch.cat(places)


def _run_cache(st):
    case = st["case"]
    fmt, out = case["fmt"], []
    pages, places = _slots(st)
    for x, stored, scales in ((st["k"], *st["cache"][:2]), (st["v"], *st["cache"][2:])):
        codes, scale = _encode(x.float(), fmt)
        stored[pages, :, places] = _store(codes, fmt)
        scales[pages, :, places] = scale
        out.append(_decode(_load(stored[pages, :, places], fmt), scales[pages, :, places],
                           fmt).to(x.dtype))
    return {"k": out[0], "v": out[1]}


def _run_attention(st):
    case = st["case"]
    H, G, D, P, fmt = (case[n] for n in ("heads", "group", "dim", "page", "fmt"))
    q, out, at = st["q"], torch.empty_like(st["q"]), 0
    for s, (n, length) in enumerate(st["sizes"]):
        pages = st["table"][s, :-(-length // P)].long()
        k, v = (_decode(_load(st["cache"][i][pages], fmt), st["cache"][i + 1][pages], fmt)
                .transpose(0, 1).reshape(H, -1, D)[:, :length] for i in (0, 2))
        hidden = torch.arange(length, device="cuda")[None, :] > \
            torch.arange(length - n, length, device="cuda")[:, None]
        for h in range(H):
            mine = q[at:at + n, h * G:(h + 1) * G].float()  # [n, G, D]
            score = (mine.reshape(n * G, D) @ k[h].t()).view(n, G, length) / math.sqrt(D)
            score = score.masked_fill(hidden[:, None, :], -math.inf)
            p = torch.exp(score - score.amax(-1, keepdim=True))
            o = p.view(n * G, length) @ v[h] / p.sum(-1).view(n * G, 1)
            out[at:at + n, h * G:(h + 1) * G] = o.view(n, G, D).to(q.dtype)
        at += n
    return {"o": out}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op, fmt, dt = case["op"], case["fmt"], TYPES[case["dtype"]]
    if op == "quantise":
        packed = _packed(state["x"], fmt)
        return {"x": _values(packed, case["cols"], fmt).to(dt), "scale": packed[1]}
    if op == "cache":
        return _run_cache(state)
    if op == "attention":
        return _run_attention(state)
    N = case["N"]
    W = _values(state["w"], N, "fp4")
    if op == "linear":
        y = _values(_packed(state["x"], fmt), N, fmt) @ W.t()
        if state["bias"] is not None:
            y = y + state["bias"]
        if state["residual"] is not None:
            y = y + state["residual"].float()
        return {"y": y.to(dt)}
    dy = state["dy"].float()
    dw = None if state["x"] is None else (dy.t() @ _values(state["x"], N, fmt)).to(dt)
    return {"dx": (dy @ W).to(dt), "dw": dw, "dbias": dy.sum(0)}


def _held(rows, cols, fmt):
    """Bytes of a quantised matrix."""
    groups = -(-cols // GROUP)
    return rows * groups * (GROUP + 1 if fmt == "fp8" else GROUP // 2 + 1)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    op, fmt = case["op"], case["fmt"]
    if op == "quantise":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * (n * size + _held(case["rows"], case["cols"], fmt)), "flops": 4 * n}
    if op in ("cache", "attention"):
        sizes = _lengths(case)
        H, G, D = case["heads"], case["group"], case["dim"]
        tokens = sum(n for n, _ in sizes)
        if op == "cache":
            moved = tokens * H * D * size + _held(tokens * H, D, fmt)
            return {"bytes": 4 * moved, "flops": 8 * tokens * H * D}
        keys = sum(length for _, length in sizes)
        pairs = sum(n * length - n * (n - 1) // 2 for n, length in sizes)
        return {"bytes": 2 * _held(keys * H, D, fmt) + 2 * tokens * H * G * D * size,
                "flops": 4 * pairs * H * G * D}
    B, M, N = case["B"], case["M"], case["N"]
    held = _held(M, N, "fp4")
    if op == "linear":
        moved = B * N * size + B * M * size * (1 + case["residual"])
        return {"bytes": held + moved + (4 * M if case["bias"] else 0), "flops": 2 * B * M * N}
    moved = B * M * size + B * N * size + 4 * M
    if case["dw"]:
        moved += _held(B, N, fmt) + M * N * size
    return {"bytes": held + moved, "flops": (4 if case["dw"] else 2) * B * M * N}


def _exact_table(fmt):
    """The format's values by code, float64: sign, exponent and mantissa bits."""
    bits, mantissa, bias = (4, 1, 1) if fmt == "fp4" else (8, 3, 7)
    values = []
    for c in range(1 << (bits - 1)):
        e, m = c >> mantissa, c & ((1 << mantissa) - 1)
        part = m / (1 << mantissa)
        values.append(part * 2.0 ** (1 - bias) if e == 0 else (1 + part) * 2.0 ** (e - bias))
    if fmt == "fp8":
        values[-1] = math.nan
    values += [-v for v in values]
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _exact_quantised(x, fmt):
    """(values, scale bytes) of x along its last dimension, float64: the nearest value of the
    format's list, the even one of two as near, found between the list's midpoints."""
    half = _exact_table(fmt)[:8 if fmt == "fp4" else 127]
    middle = (half[1:] + half[:-1]) / 2
    powers = torch.tensor([2.0 ** (e - 127) for e in range(255)], dtype=torch.float64,
                          device="cuda")
    out, scales = torch.empty(x.shape, dtype=torch.float64, device="cuda"), []
    for c in range(0, x.shape[-1], GROUP):
        v = x[..., c:c + GROUP].double()
        top = v.abs().amax(-1)
        # frexp: top = m 2^p with m in [1/2, 1), so floor(log2 top) = p - 1
        p = torch.frexp(top)[1].long() - 1
        e = torch.where(top < 2.0 ** -126, torch.zeros_like(p), p + 127 - TOP[fmt]).clamp_min(0)
        step = powers[e].unsqueeze(-1)
        u = v.abs() / step
        low = torch.searchsorted(middle, u.contiguous())  # midpoints below u
        tie = (low < middle.numel()) & (u == middle[low.clamp_max(middle.numel() - 1)])
        low = torch.where(tie & (low % 2 == 1), low + 1, low)
        out[..., c:c + GROUP] = torch.copysign(half[low] * step, v)
        scales.append(e)
    return out, torch.stack(scales, -1).to(torch.uint8)


def _exact_values(stored, scale, fmt):
    """Values of stored codes, float64."""
    table = _exact_table(fmt)
    powers = torch.tensor([2.0 ** (e - 127) for e in range(255)] + [math.nan],
                          dtype=torch.float64, device=stored.device)
    v = torch.empty(*stored.shape[:-1], scale.shape[-1] * GROUP, dtype=torch.float64,
                    device=stored.device)
    if fmt == "fp8":
        v.copy_(table[stored.int()])
    else:
        v[..., 0::2] = table[(stored % 16).int()]
        v[..., 1::2] = table[torch.div(stored, 16, rounding_mode="floor").int()]
    return v * powers[scale.int()].repeat_interleave(GROUP, -1)


def exact(case, seed):
    st = prepare(case, seed)
    op, fmt = case["op"], case["fmt"]
    if op == "quantise":
        v, scale = _exact_quantised(st["x"], fmt)
        return {"x": v, "scale": scale}
    if op == "cache":
        return {n: _exact_quantised(st[n], fmt)[0] for n in ("k", "v")}
    if op == "attention":
        return {"o": _exact_attention(st)}
    N = case["N"]
    W = _exact_values(*st["w"], "fp4")[:, :N]
    if op == "linear":
        x = _exact_quantised(st["x"], fmt)[0]
        y = torch.matmul(x, W.t().contiguous())
        if case["bias"]:
            y += st["bias"].double()[None, :]
        if case["residual"]:
            y += st["residual"].double()
        return {"y": y}
    dy = st["dy"].double()
    dw = None
    if case["dw"]:
        dw = torch.matmul(dy.t().contiguous(), _exact_values(*st["x"], fmt)[:, :N].contiguous())
    return {"dx": torch.matmul(dy, W.contiguous()), "dw": dw, "dbias": dy.sum(0)}


def _exact_attention(st):
    case = st["case"]
    G, D, P, fmt = case["group"], case["dim"], case["page"], case["fmt"]
    kc, ks, vc, vs = st["cache"]
    out, at = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"), 0
    for s, (n, length) in enumerate(st["sizes"]):
        t = torch.arange(length, device="cuda")
        page, place = st["table"][s].long()[t // P], t % P
        last = t[length - n:]
        for h in range(case["heads"]):
            k = _exact_values(kc[page, h, place], ks[page, h, place], fmt)
            v = _exact_values(vc[page, h, place], vs[page, h, place], fmt)
            kt = k.t().contiguous()
            for g in range(h * G, (h + 1) * G):
                for i in range(0, n, 2048):
                    rows = slice(at + i, at + min(n, i + 2048))
                    z = torch.matmul(st["q"][rows, g].double(), kt) * D ** -0.5
                    z[t[None, :] > last[i:i + 2048, None]] = -math.inf
                    out[rows, g] = torch.matmul(torch.softmax(z, -1), v)
        at += n
    return out
