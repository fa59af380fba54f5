"""The dense operators around the trellis codec, as measured cases.

  quantize  rows to 8-bit integers with one scale a row (activations: a token a row)
  decode    a matrix's 16x16-tile streams to rows of 8-bit integers, one scale a row (channel)
  linear8   product of two 8-bit matrices with a scale for each token and each channel
  gated     h = act(x Wg^T) * (x Wu^T), both projections and their product
  gated_vjp its gradients: x, Wg and Wu, from the upstream gradient and the saved projections

`run` computes them in plain torch operations, or, where `own` is true, calls the
framework.  `exact` is the same in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "i8": 1}


def listed():
    return [
        # one token's activations before an 8-bit projection: launch latency
        {"name": "quantize 1x8192 bf16", "op": "quantize", "rows": 1, "cols": 8192, "dtype": "bf16"},
        # a prefill's hidden activations before the down projection: bandwidth
        {"name": "quantize 4096x14336 bf16", "op": "quantize", "rows": 4096, "cols": 14336, "dtype": "bf16"},
        # one square projection's streams to 8-bit rows, tail-biting 1MAD
        {"name": "decode 4096x4096 1mad tb", "op": "decode", "M": 4096, "N": 4096, "code": "1mad", "tailbiting": True},
        # the largest matrix of the decode benchmarks, plain 3INST streams
        {"name": "decode 28672x8192 3inst", "op": "decode", "M": 28672, "N": 8192, "code": "3inst", "tailbiting": False},
        # one token through a square projection: latency and the weights' bytes
        {"name": "linear8 1x4096x4096 bf16", "op": "linear8", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16"},
        # a ragged batch of decoding sequences through a wide down projection
        {"name": "linear8 77x8192x28672 f16", "op": "linear8", "M": 77, "N": 8192, "K": 28672, "dtype": "f16"},
        # a prefill through a wide up projection
        {"name": "linear8 4096x28672x8192 bf16", "op": "linear8", "M": 4096, "N": 28672, "K": 8192, "dtype": "bf16"},
        # one token through a gated feed-forward's first half
        {"name": "gated 1x14336x4096 bf16", "op": "gated", "M": 1, "F": 14336, "K": 4096, "dtype": "bf16", "act": "silu"},
        # odd sizes: rows that are no multiple of any vector width
        {"name": "gated 333x2731x1001 f16", "op": "gated", "M": 333, "F": 2731, "K": 1001, "dtype": "f16", "act": "gelu_tanh"},
        # a training micro-batch, forward
        {"name": "gated 4096x14336x4096 bf16", "op": "gated", "M": 4096, "F": 14336, "K": 4096, "dtype": "bf16", "act": "silu"},
        # a short fine-tuning batch, backward
        {"name": "gated_vjp 120x14336x4096 f16", "op": "gated_vjp", "M": 120, "F": 14336, "K": 4096, "dtype": "f16", "act": "gelu"},
        # a training micro-batch, backward
        {"name": "gated_vjp 4096x14336x4096", "op": "gated_vjp", "M": 4096, "F": 14336, "K": 4096, "dtype": "bf16", "act": "silu"},
    ]


def draw(rng):
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        step = rng.choice([1, 8, 16, 64, 128])     # any size, or one of the usual multiples
        return max(lo, min(hi, n // step * step))

    def tokens():
        return rng.choice([1, size(1, 32), size(16, 512), size(256, 4096)])

    op = rng.choice(["quantize", "decode", "linear8", "gated", "gated_vjp"])
    if op == "quantize":
        return {"op": op, "rows": tokens(), "cols": size(64, 28672) if rng.random() < 0.5 else size(1024, 14336),
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op == "decode":
        return {"op": op, "M": 16 * size(4, 1792), "N": 16 * size(4, 512), "code": rng.choice(["1mad", "3inst", "xor"]),
                "tailbiting": rng.random() < 0.5}
    dtype = rng.choice(["bf16", "f16"])
    if op == "linear8":
        return {"op": op, "M": tokens(), "N": size(64, 28672), "K": size(64, 8192),
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    return {"op": op, "M": tokens(), "F": size(64, 14336), "K": size(64, 4096), "dtype": dtype,
            "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])}


XOR_MASKS = (0x2D35, 0x1ACB, 0x34AE, 0x0F53)     # the parity masks of the framework's workloads
XOR_PALETTES = ((-6.0, -1.5, 0.0, 2.0), (-4.0, -1.0, 0.5, 3.0), (-3.0, -0.5, 1.0, 4.0), (-2.0, 0.0, 1.5, 6.0))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def activations(rows, cols):
        # a few channels of activations are many times larger than the others
        big = torch.rand(cols, generator=g, device="cuda") < 0.01
        return normal(rows, cols) * torch.where(big, 8.0, 1.0)

    s = dict(case)
    op = case["op"]
    if op == "quantize":
        s["x"] = activations(case["rows"], case["cols"]).to(DTYPES[case["dtype"]])
        return s
    if op == "decode":
        words = 16 if case["tailbiting"] else 17
        n = (case["M"] // 16) * (case["N"] // 16)
        bits = torch.randint(-2 ** 31, 2 ** 31, (n, words), generator=g, device="cuda", dtype=torch.int64)
        if not case["tailbiting"]:
            bits[:, 16] &= 0xFFFC0000             # 526 stream bits: the last word holds 14 of them
        s["bits"] = bits.to(torch.int32)
        return s
    dt = DTYPES[case["dtype"]]
    if op == "linear8":
        def ints(r, c):
            return (normal(r, c) * 32.0).round().clamp(-127, 127).to(torch.int8)
        s["a"], s["w"] = ints(case["M"], case["K"]), ints(case["N"], case["K"])
        s["a_scale"] = torch.rand(case["M"], generator=g, device="cuda") * 0.05 + 0.01
        s["w_scale"] = (torch.rand(case["N"], generator=g, device="cuda") * 0.05 + 0.01) / math.sqrt(case["K"])
        return s
    M, F, K = case["M"], case["F"], case["K"]
    x = normal(M, K)
    s["x"] = x.to(dt)
    s["w_gate"] = (normal(F, K) / math.sqrt(K)).to(dt)
    s["w_up"] = (normal(F, K) / math.sqrt(K)).to(dt)
    if op == "gated_vjp":
        # what the forward pass saved, and the gradient that comes back to it
        s["gate"] = (s["x"].float() @ s["w_gate"].float().t()).to(dt)
        s["up"] = (s["x"].float() @ s["w_up"].float().t()).to(dt)
        s["grad_h"] = (normal(M, F) * 0.1).to(dt)
    return s


# ---- plain forms ------------------------------------------------------------------------------

def plain_quantize(x):
    x = x.float()
    # the quotients decide at half steps: 64 bits
    scale = (x.abs().amax(1).double() / 127.0).float()
    q = torch.round(x.double() / scale.double()[:, None]).clamp(-127, 127)
    return torch.where(scale[:, None] > 0, q, 0.0).to(torch.int8), scale


def plain_windows(bits, tailbiting):
    """The 16-bit states of the 256 weights of every stream, int64 [streams][256]."""
    w = bits.to(torch.int64) & 0xFFFFFFFF
    following = torch.cat([w[:, 1:], w[:, :1]], 1) if tailbiting else torch.cat([w[:, 1:], w[:, :1] * 0], 1)
    pair = (w << 16) | (following >> 16)                       # 48 bits from each word's start
    pair = pair[:, :16]
    shift = torch.arange(16, device=bits.device) * 2
    return ((pair[:, :, None] >> (32 - shift)) & 0xFFFF).reshape(bits.shape[0], 256)


def plain_parity(v):
    v = v ^ (v >> 8)
    v = v ^ (v >> 4)
    v = v ^ (v >> 2)
    return (v ^ (v >> 1)) & 1


def plain_code(x, code):
    if code == "xor":
        h = x >> 2
        p = [plain_parity(h & m) for m in XOR_MASKS]
        entry = (x & 3) ^ (2 * p[2] + p[3])
        return torch.tensor(XOR_PALETTES, device=x.device)[2 * p[0] + p[1], entry]
    u = (x * 34038481 + 76625530) & 0xFFFFFFFF
    if code == "1mad":
        total = (u & 255) + ((u >> 8) & 255) + ((u >> 16) & 255) + (u >> 24)
        return ((total - 510).double() / 147.8).float()
    v = ((u & 0x8FFF8FFF) ^ 0x3B603B60).to(torch.int32)
    half = v.view(torch.float16).reshape(*v.shape, 2)
    return ((half[..., 0] + half[..., 1]).double() / 1.244).float()


def plain_decode(bits, M, N, code, tailbiting):
    w = plain_code(plain_windows(bits, tailbiting), code)
    w = w.reshape(M // 16, N // 16, 16, 16).permute(0, 2, 1, 3).reshape(M, N)
    return plain_quantize(w)


def plain_linear8(a, a_scale, w, w_scale, dt):
    # sums of products of integers: exact in 32-bit floating point while they stay below 2^24
    return ((a.float() @ w.float().t()) * a_scale[:, None] * w_scale).to(dt)


def plain_act(g, act):
    if act == "relu":
        return g.clamp(min=0)
    if act == "gelu":
        return g * 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return g * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    s = 1 / (1 + torch.exp(-g))
    return s if act == "sigmoid" else g * s


def plain_act_grad(g, act):
    if act == "relu":
        return (g > 0).to(g.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
        return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
    s = 1 / (1 + torch.exp(-g))
    return s * (1 - s) if act == "sigmoid" else s * (1 + g * (1 - s))


def plain_gated(x, w_gate, w_up, act):
    x32 = x.float()
    gate, up = x32 @ w_gate.float().t(), x32 @ w_up.float().t()
    return (plain_act(gate, act) * up).to(x.dtype)


def plain_gated_vjp(x, w_gate, w_up, gate, up, grad_h, act):
    g, u, d, x32 = gate.float(), up.float(), grad_h.float(), x.float()
    d_gate, d_up = d * u * plain_act_grad(g, act), d * plain_act(g, act)
    grad_x = d_gate @ w_gate.float() + d_up @ w_up.float()
    return grad_x.to(x.dtype), (d_gate.t() @ x32).to(x.dtype), (d_up.t() @ x32).to(x.dtype)


def run(s):
    op = s["op"]
    if own:
        from trellis_coded_weight_amd import api
        if op == "quantize":
            return api.quantize_rows(s["x"])
        if op == "decode":
            code = ("xor", XOR_MASKS) if s["code"] == "xor" else s["code"]
            return api.decode_matrix(s["bits"], s["M"], s["N"], L=16, k=2, code=code, tailbiting=s["tailbiting"],
                                     dtype=torch.int8)
        if op == "linear8":
            return api.matmul_int8(s["a"], s["a_scale"], s["w"], s["w_scale"], dtype=DTYPES[s["dtype"]])
        if op == "gated":
            return api.gated(s["x"], s["w_gate"], s["w_up"], activation=s["act"])
        return api.gated_vjp(s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], s["grad_h"], activation=s["act"])
    if op == "quantize":
        return plain_quantize(s["x"])
    if op == "decode":
        return plain_decode(s["bits"], s["M"], s["N"], s["code"], s["tailbiting"])
    if op == "linear8":
        return plain_linear8(s["a"], s["a_scale"], s["w"], s["w_scale"], DTYPES[s["dtype"]])
    if op == "gated":
        return plain_gated(s["x"], s["w_gate"], s["w_up"], s["act"])
    return plain_gated_vjp(s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], s["grad_h"], s["act"])


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (BYTES[case["dtype"]] + 1) + 4 * case["rows"], "flops": 3 * n}
    if op == "decode":
        n = case["M"] * case["N"]
        # 2 bits a weight in, 8 bits out; window, code, scale and rounding
        return {"bytes": n // 256 * (64 if case["tailbiting"] else 68) + n + 4 * case["M"], "flops": 8 * n}
    if op == "linear8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K + 4) + M * N * BYTES[case["dtype"]], "flops": 2 * M * N * K}
    M, F, K = case["M"], case["F"], case["K"]
    if op == "gated":
        return {"bytes": 2 * (M * K + 2 * F * K + M * F), "flops": 4 * M * F * K}
    return {"bytes": 2 * (2 * M * K + 4 * F * K + 3 * M * F), "flops": 8 * M * F * K}


# ---- the same from the definitions, in 64 bits -------------------------------------------------

def exact_rows_to_int8(v):
    """Symmetric 8-bit rows of the 64-bit matrix v: the scale is the row's largest magnitude over
    127, held in 32 bits; each value is the nearest whole multiple of it, halves to even."""
    scale = (v.abs().max(dim=1).values / 127).float()
    s = scale.double().unsqueeze(1)
    q = torch.where(s == 0, torch.zeros_like(v), v / s)
    return torch.round(q).clip(-127, 127).to(torch.int8), scale


def exact_codebook(code):
    x = np.arange(65536, dtype=np.uint64)
    u = (x * np.uint64(34038481) + np.uint64(76625530)).astype(np.uint32)
    if code == "1mad":
        v = (u.view(np.uint8).reshape(-1, 4).astype(np.float64).sum(1) - 510) / 147.8
    elif code == "3inst":
        h = ((u & np.uint32(0x8FFF8FFF)) ^ np.uint32(0x3B603B60)).view(np.float16).reshape(-1, 2)
        v = np.add(h[:, 0], h[:, 1], dtype=np.float16).astype(np.float64) / 1.244
    else:
        bit = [np.array([bin((k >> 2) & m).count("1") % 2 for k in range(65536)]) for m in XOR_MASKS]
        v = np.array(XOR_PALETTES)[bit[0] * 2 + bit[1], (x.astype(np.int64) % 4) ^ (bit[2] * 2 + bit[3])]
    # a code value is held in 32 bits: one rounding of the 64-bit quotient
    return torch.from_numpy(v.astype(np.float32).astype(np.float64)).cuda()


def exact_activation(t, act):
    """The activation and its derivative."""
    if act == "relu":
        on = t > 0
        return torch.where(on, t, torch.zeros_like(t)), on.double()
    if act == "gelu":
        normal = 0.5 * torch.special.erfc(-t / math.sqrt(2.0))
        return t * normal, normal + t * torch.exp(-t.square() / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(8 / math.pi)                            # (1 + tanh z) / 2 = sigmoid(2 z)
        s = torch.sigmoid(c * (t + 0.044715 * t ** 3))
        return t * s, s + t * s * (1 - s) * c * (1 + 0.134145 * t ** 2)
    s = torch.sigmoid(t)
    slope = s * torch.sigmoid(-t)
    return (s, slope) if act == "sigmoid" else (t * s, s + t * slope)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return exact_rows_to_int8(s["x"].double())
    if op == "decode":
        M, N = case["M"], case["N"]
        book = exact_codebook(case["code"])
        out = []
        per = max(1, (1 << 24) // N // 16)                    # bands of 16 rows at a time
        streams = s["bits"].reshape(M // 16, N // 16, -1)
        for lo in range(0, M // 16, per):
            words = streams[lo:lo + per]
            pos = torch.arange(31, -1, -1, device="cuda", dtype=torch.int32)
            stream = ((words.unsqueeze(-1) >> pos) & 1).flatten(2)                # every bit in order
            if case["tailbiting"]:
                stream = torch.cat([stream, stream[..., :14]], -1)
            state = torch.zeros(*stream.shape[:2], 256, dtype=torch.int64, device="cuda")
            for b in range(16):
                state = 2 * state + stream[..., b:b + 511:2]
            v = book[state].unflatten(-1, (16, 16)).transpose(1, 2).flatten(2).flatten(0, 1)
            out.append(exact_rows_to_int8(v))
        return torch.cat([q for q, _ in out]), torch.cat([c for _, c in out])
    if op == "linear8":
        acc = torch.mm(s["a"].double(), s["w"].double().t())
        return torch.outer(s["a_scale"].double(), s["w_scale"].double()).mul_(acc)
    x, wg, wu = s["x"].double(), s["w_gate"].double(), s["w_up"].double()
    if op == "gated":
        y, _ = exact_activation(torch.mm(x, wg.t()), case["act"])
        return y.mul_(torch.mm(x, wu.t()))
    y, slope = exact_activation(s["gate"].double(), case["act"])
    dh = s["grad_h"].double()
    du = dh * y
    dg = dh * s["up"].double() * slope
    # one product over both halves of the feed-forward's width
    return torch.mm(torch.cat([dg, du], 1), torch.cat([wg, wu], 0)), torch.mm(dg.t(), x), torch.mm(du.t(), x)
