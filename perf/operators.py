"""The coded linear layer's operators, as they are measured: the batched product with a
trellis-coded matrix (decoded inside the call) with row scale, bias, activation and
residual; its backward pass from 8-bit checkpoints; and the checkpoints themselves.

Weights come as random bitstreams with start states below 2^(L - kV): every such stream
is a path of the trellis, and with a Gaussian-quantile codebook it decodes to N(0, 1)
weights, as an encoder's output does.  The row scale brings the layer's output to unit size.
"""
import math

import torch

own = False  # False: plain torch forms; True: the framework's operators

GROUP = 32  # values that share one scale in a checkpoint

# (L, k, V, T) of the repository's workloads and tests
TRELLISES = ((16, 2, 1, 256), (16, 3, 1, 256), (16, 2, 2, 256), (8, 2, 1, 64), (12, 2, 1, 64))
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "silu", "gelu")
LARGEST = 8192 * 4096 * 14336  # B M N of the largest product listed


def _linear(name, B, M, N, trellis, dtype, act="none", bias=False, residual=False, pre=False):
    L, k, V, T = trellis
    return {"name": name, "op": "linear", "B": B, "M": M, "N": N, "L": L, "k": k, "V": V,
            "T": T, "dtype": dtype, "act": act, "bias": bias, "residual": residual,
            "pre": pre}


def _backward(name, B, M, N, trellis, dtype, act="none", dw=True):
    L, k, V, T = trellis
    return {"name": name, "op": "backward", "B": B, "M": M, "N": N, "L": L, "k": k, "V": V,
            "T": T, "dtype": dtype, "act": act, "dw": dw}


def _checkpoint(name, B, N, dtype):
    return {"name": name, "op": "checkpoint", "B": B, "N": N, "dtype": dtype}


def listed():
    return [
        # one token through a 1B-class projection: latency
        _linear("token-2048", 1, 2048, 2048, TRELLISES[0], "bf16", residual=True),
        # one token through an 8B-class up projection, two weights a step
        _linear("token-mlp-V2", 1, 14336, 4096, TRELLISES[2], "f16", act="silu"),
        # a batch of sequences, one token each, through the 3-bit down projection
        _linear("tokens16-down-k3", 16, 4096, 14336, TRELLISES[1], "bf16", residual=True),
        # drafted or ragged tokens of some sequences, with bias and gelu
        _linear("tokens100-4096", 100, 4096, 4096, TRELLISES[0], "bf16", act="gelu", bias=True),
        # a training step's forward in 32 bits at an odd batch, its pre-activation kept
        _linear("train-f32-333", 333, 2048, 2048, TRELLISES[0], "f32", act="relu", bias=True,
                pre=True),
        # a prompt through the up projection, pre-activation kept for the backward pass
        _linear("prompt-mlp-V2", 2048, 14336, 4096, TRELLISES[2], "bf16", act="silu", pre=True),
        # a long prompt through the 3-bit down projection: the largest product
        _linear("prompt-down-k3", 8192, 4096, 14336, TRELLISES[1], "bf16", residual=True),
        # fine-tuning steps: gradients of input, matrix and bias from 8-bit checkpoints
        _backward("grad-2048", 509, 2048, 2048, TRELLISES[0], "bf16", act="gelu"),
        _backward("grad-4096", 4096, 4096, 4096, TRELLISES[0], "f16", act="silu"),
        # the matrix frozen, 32-bit training: the input's gradient alone
        _backward("grad-f32-dx", 1000, 2048, 2048, TRELLISES[0], "f32", dw=False),
        # activations kept in 8 bits and read back: a short sequence, and a long one's MLP
        _checkpoint("keep-500x2048", 500, 2048, "bf16"),
        _checkpoint("keep-16384x14336", 16384, 14336, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear", "backward", "backward", "checkpoint"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "checkpoint":
        case = _checkpoint("", _log_int(rng, 1, 16384), _log_int(rng, 33, 14336), dtype)
    else:
        trellis = rng.choice(TRELLISES)
        T = trellis[3]
        M = _log_int(rng, 64, 14336)
        N = T * _log_int(rng, 1, 14336 // T)
        products = 1 if op == "linear" else 2
        B = _log_int(rng, 1, min(16384, max(1, LARGEST // (products * M * N))))
        act = rng.choice(ACTS)
        if op == "linear":
            case = _linear("", B, M, N, trellis, dtype, act, rng.random() < 0.5,
                           rng.random() < 0.5, rng.random() < 0.3)
        else:
            case = _backward("", B, M, N, trellis, dtype, act, rng.random() < 0.7)
    del case["name"]
    return case


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _power_of_two(e):
    """2^e exactly, float64, for integers |e| < 1000."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _pack(x):
    """Plain form of the checkpoint: (codes int8 [B, N], scale bytes [B, ceil(N / 32)])."""
    B, N = x.shape
    groups = (N + GROUP - 1) // GROUP
    v = torch.zeros(B, groups * GROUP, dtype=torch.float64, device=x.device)
    v[:, :N] = x.double()
    v = v.view(B, groups, GROUP)
    top = v.abs().amax(2)
    # exponent field of the largest magnitude as a 32-bit float
    e = (top.float().view(torch.int32) >> 23) & 255
    q = torch.clamp(torch.round(v * _power_of_two(133 - e).unsqueeze(2)), -127, 127)
    q = torch.where((e == 255).unsqueeze(2), torch.zeros_like(q), q)
    return q.view(B, -1)[:, :N].to(torch.int8).contiguous(), e.to(torch.uint8)


def _unpack(codes, scale):
    """Plain form: the float32 values that codes and scale bytes stand for."""
    N = codes.shape[1]
    e = scale.to(torch.int32).repeat_interleave(GROUP, 1)[:, :N]
    v = codes.double() * _power_of_two(e - 133)
    v = torch.where(e == 255, torch.full_like(v, float("nan")), v)
    return v.float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]
    B, N = case["B"], case["N"]
    st = {"case": case}
    if case["op"] == "checkpoint":
        # activations: most of them small, a few channels far larger than the others
        channel = torch.exp(_randn(g, 1, N))
        st["x"] = (_randn(g, B, N) * channel).to(dt)
        return st
    M, L, k, V, T = (case[n] for n in ("M", "L", "k", "V", "T"))
    nb, nw = M * (N // T), (k * T + 31) // 32
    bits = torch.randint(-2 ** 31, 2 ** 31, (nb, nw), generator=g, device="cuda",
                         dtype=torch.int64).to(torch.int32)
    tail = k * T % 32
    if tail:  # unused tail bits are zero
        bits[:, -1] &= -(1 << (32 - tail))
    st["bits"] = bits
    st["s0"] = torch.randint(0, 1 << (L - k * V), (nb,), generator=g, device="cuda",
                             dtype=torch.int32)
    # Gaussian quantiles in a shuffled order, rounded once to the layer's type
    j = torch.arange(1 << L, device="cuda", dtype=torch.float64)
    quantile = math.sqrt(2.0) * torch.erfinv((2.0 * j + 1.0) / (1 << L) - 1.0)
    st["table"] = torch.stack([quantile[torch.randperm(1 << L, generator=g, device="cuda")]
                               for _ in range(V)], 1).to(dt).contiguous()
    st["row_scale"] = torch.exp(0.3 * _randn(g, M)) / math.sqrt(N)
    if case["op"] == "linear":
        st["x"] = _randn(g, B, N).to(dt)
        st["bias"] = _randn(g, M) if case["bias"] else None
        st["residual"] = _randn(g, B, M).to(dt) if case["residual"] else None
    else:
        st["dy"] = _randn(g, B, M).to(dt)
        st["z"] = _pack(_randn(g, B, M).to(dt)) if case["act"] != "none" else None
        st["x"] = _pack(_randn(g, B, N).to(dt)) if case["dw"] else None
    return st


def _decode(st):
    """Plain form of the decode, float32 [M, N]: step t's state is the L-bit window of
    s_0 || b_1 || ... that ends with b_t, read from two neighbouring 32-bit words."""
    case = st["case"]
    M, N, L, k, V, T = (case[n] for n in ("M", "N", "L", "k", "V", "T"))
    words = torch.cat([st["s0"].view(-1, 1), st["bits"]], 1).long() & 0xFFFFFFFF
    end = torch.arange(1, T // V + 1, device=words.device) * (k * V)
    last = (end - 1) // 32
    both = (words[:, last] << 32) | words[:, last + 1]
    state = (both >> (32 * (last + 1) - end)) & ((1 << L) - 1)
    return st["table"].float()[state.view(-1)].view(M, N)


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + \
            z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _run_own(st):
    from trellis_coded_bit_amd import api
    case = st["case"]
    if case["op"] == "checkpoint":
        packed = api.act_pack(st["x"])
        return {"x": api.act_unpack(packed, st["x"].dtype), "scale": packed.scale}
    shape = [case[n] for n in ("M", "N", "L", "k", "V", "T")]
    if case["op"] == "linear":
        y = api.decode_linear(st["bits"], st["s0"], st["table"], st["x"], *shape,
                              row_scale=st["row_scale"], bias=st["bias"], act=case["act"],
                              residual=st["residual"], pre=case["pre"])
        return {"y": y[0], "z": y[1]} if case["pre"] else {"y": y}
    z = None if st["z"] is None else api.Packed(*st["z"])
    x = None if st["x"] is None else api.Packed(*st["x"])
    dx, dw, dbias = api.decode_linear_backward(st["bits"], st["s0"], st["table"], st["dy"],
                                               *shape, row_scale=st["row_scale"],
                                               act=case["act"], z=z, x=x)
    return {"dx": dx, "dw": dw, "dbias": dbias}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    dt = TYPES[case["dtype"]]
    if case["op"] == "checkpoint":
        codes, scale = _pack(state["x"])
        return {"x": _unpack(codes, scale).to(dt), "scale": scale}
    W = _decode(state)
    if case["op"] == "linear":
        z = (state["x"].float() @ W.t()) * state["row_scale"]
        if state["bias"] is not None:
            z = z + state["bias"]
        y = _act(z, case["act"])
        if state["residual"] is not None:
            y = y + state["residual"].float()
        return {"y": y.to(dt), "z": z.to(dt)} if case["pre"] else {"y": y.to(dt)}
    grad = state["dy"].float()
    if state["z"] is not None:
        grad = grad * _act_grad(_unpack(*state["z"]), case["act"])
    dbias = grad.sum(0)
    grad = grad * state["row_scale"]
    dx = (grad @ W).to(dt)
    dw = None if state["x"] is None else (grad.t() @ _unpack(*state["x"])).to(dt)
    return {"dx": dx, "dw": dw, "dbias": dbias}


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    B, N = case["B"], case["N"]
    if case["op"] == "checkpoint":
        held = B * N + B * ((N + GROUP - 1) // GROUP)
        return {"bytes": 2 * (B * N * size + held), "flops": 4 * B * N}
    M, L, k, V, T = (case[n] for n in ("M", "L", "k", "V", "T"))
    blocks = M * (N // T)
    streams = blocks * (4 * ((k * T + 31) // 32) + 4) + (1 << L) * V * size + 4 * M
    if case["op"] == "linear":
        moved = B * N * size + B * M * size * (1 + case["residual"] + case["pre"])
        moved += 4 * M if case["bias"] else 0
        return {"bytes": streams + moved, "flops": 2 * B * M * N}
    moved = B * M * size + B * N * size + 4 * M
    if case["act"] != "none":
        moved += B * M + B * ((M + GROUP - 1) // GROUP)
    if case["dw"]:
        moved += B * N + B * ((N + GROUP - 1) // GROUP) + M * N * size
    return {"bytes": streams + moved, "flops": (4 if case["dw"] else 2) * B * M * N}


def _exact_values(codes, scale):
    B, N = codes.shape
    powers = torch.tensor([2.0 ** (e - 133) for e in range(255)] + [math.nan],
                          dtype=torch.float64, device=codes.device)
    group = torch.arange(N, device=codes.device) // GROUP
    return codes.double() * powers[scale.long()][:, group]


def _exact_weights(st):
    """The shift register itself, step by step: s = (s << kV | b_t) mod 2^L."""
    case = st["case"]
    M, N, L, k, V, T = (case[n] for n in ("M", "N", "L", "k", "V", "T"))
    kv = k * V
    shifts = torch.arange(31, -1, -1, device="cuda")
    s = st["s0"].long()
    out = torch.empty(s.numel(), T // V, V, dtype=torch.float64, device="cuda")
    table = st["table"].double()
    for t in range(T // V):
        for b in range(t * kv, (t + 1) * kv):  # the chunk's bits, most significant first
            bit = (st["bits"][:, b // 32].long() >> shifts[b % 32]) & 1
            s = ((s << 1) | bit) & ((1 << L) - 1)
        out[:, t] = table[s]
    return out.view(M, N)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "checkpoint":
        x = st["x"].double()
        out, scales = torch.empty_like(x), []
        powers = torch.tensor([2.0 ** (p - 146) for p in range(280)], dtype=torch.float64,
                              device="cuda")
        for c in range(0, case["N"], GROUP):
            v = x[:, c:c + GROUP]
            top = v.abs().amax(1, keepdim=True)
            # frexp: top = m 2^p with m in [1/2, 1), so floor(log2 top) = p - 1
            p = torch.frexp(top)[1].long() - 1
            p = torch.where(top < 2.0 ** -126, torch.full_like(p, -127), p)
            step = powers[p + 140]
            out[:, c:c + GROUP] = torch.clamp(torch.round(v / step), -127, 127) * step
            scales.append(p + 127)
        return {"x": out, "scale": torch.cat(scales, 1).to(torch.uint8)}
    W = _exact_weights(st)
    a = st["row_scale"].double()
    if case["op"] == "linear":
        z = torch.matmul(st["x"].double(), W.t().contiguous()) * a[None, :]
        if case["bias"]:
            z = z + st["bias"].double()[None, :]
        if case["act"] == "relu":
            y = torch.where(z > 0, z, torch.zeros_like(z))
        elif case["act"] == "silu":
            y = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            y = 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
        else:
            y = z
        if case["residual"]:
            y = y + st["residual"].double()
        return {"y": y, "z": z} if case["pre"] else {"y": y}
    grad = st["dy"].double()
    if case["act"] != "none":
        z = _exact_values(*st["z"])
        if case["act"] == "relu":
            grad = torch.where(z > 0, grad, torch.zeros_like(grad))
        elif case["act"] == "silu":
            s = torch.sigmoid(z)
            grad = grad * (s + z * s * torch.sigmoid(-z))
        else:
            density = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
            grad = grad * (0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * density)
    dbias = grad.sum(0)
    grad = grad * a[None, :]
    dx = torch.matmul(grad, W)
    dw = torch.matmul(grad.t().contiguous(), _exact_values(*st["x"])) if case["dw"] else None
    return {"dx": dx, "dw": dw, "dbias": dbias}
