"""Operators of a model on coded weights, as measured cases: 8-bit floating point with block
scales, layer norm, and the distillation that trains the weights.

  blocks          rows to e4m3 with a float32 scale for each block of 128 columns of a row
                  (activations) or of 128 x 128 elements (weights)
  linear_fp8      product of two e4m3 matrices with such scales
  layer_norm      rows normalised, scaled and shifted
  layer_norm_vjp  its gradients: x, weight and bias
  distill         divergence of a model's distribution over the vocabulary from a teacher's,
                  given by its top logits: a loss a token and, in training, the logits' gradient

`run` computes them in plain torch operations, or, where `own` is true, calls the
framework.  `exact` is the same in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # one token's activations before an fp8 projection: launch latency
        {"name": "blocks 1x8192 bf16", "op": "blocks", "rows": 1, "cols": 8192, "dtype": "bf16", "block_rows": 1},
        # the largest decoded matrix of the decode benchmarks, once when a model is loaded or
        # after each update of its weights in training
        {"name": "blocks 28672x8192 bf16 square", "op": "blocks", "rows": 28672, "cols": 8192, "dtype": "bf16", "block_rows": 128},
        # one token through a square projection: latency and the weights' bytes
        {"name": "linear_fp8 1x4096x4096 bf16", "op": "linear_fp8", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16"},
        # a ragged batch of decoding sequences through a down projection
        {"name": "linear_fp8 93x8192x14336 f16", "op": "linear_fp8", "M": 93, "N": 8192, "K": 14336, "dtype": "f16"},
        # a prefill through a wide up projection
        {"name": "linear_fp8 4096x28672x8192 bf16", "op": "linear_fp8", "M": 4096, "N": 28672, "K": 8192, "dtype": "bf16"},
        # a few decoding sequences ahead of a projection
        {"name": "layer_norm 7x4096 bf16", "op": "layer_norm", "rows": 7, "cols": 4096, "dtype": "bf16", "weight": "bf16", "save": False},
        # a training micro-batch, forward
        {"name": "layer_norm 8192x8192 bf16", "op": "layer_norm", "rows": 8192, "cols": 8192, "dtype": "bf16", "weight": "f32", "save": True},
        # odd sizes in full precision, backward
        {"name": "layer_norm_vjp 333x2731 f32", "op": "layer_norm_vjp", "rows": 333, "cols": 2731, "dtype": "f32", "weight": "f32"},
        # a training micro-batch, backward
        {"name": "layer_norm_vjp 8192x8192 bf16", "op": "layer_norm_vjp", "rows": 8192, "cols": 8192, "dtype": "bf16", "weight": "f32"},
        # a few tokens scored against the teacher: rows too few to fill the chip by themselves
        {"name": "distill 16x128000 bf16 loss", "op": "distill", "rows": 16, "vocab": 128000, "k": 64, "dtype": "bf16", "teacher": "f32", "tau": 1.0, "grad": False},
        # a fine-tuning batch over a vocabulary of no even size
        {"name": "distill 1001x50021 f16", "op": "distill", "rows": 1001, "vocab": 50021, "k": 20, "dtype": "f16", "teacher": "f16", "tau": 2.0, "grad": True},
        # a training micro-batch over a wide vocabulary
        {"name": "distill 4096x128000 bf16", "op": "distill", "rows": 4096, "vocab": 128000, "k": 64, "dtype": "bf16", "teacher": "f32", "tau": 1.0, "grad": True},
    ]


def draw(rng):
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        step = rng.choice([1, 8, 16, 64, 128])     # any size, or one of the usual multiples
        return max(lo, min(hi, n // step * step))

    def tokens():
        return rng.choice([1, size(1, 32), size(16, 512), size(256, 4096)])

    op = rng.choice(["blocks", "linear_fp8", "linear_fp8", "layer_norm", "layer_norm_vjp", "distill", "distill"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "blocks":
        if rng.random() < 0.5:
            return {"op": op, "rows": tokens(), "cols": size(64, 28672), "dtype": dtype, "block_rows": 1}
        return {"op": op, "rows": size(64, 28672), "cols": size(64, 4096), "dtype": dtype, "block_rows": 128}
    if op == "linear_fp8":
        return {"op": op, "M": tokens(), "N": size(64, 28672), "K": size(64, 8192), "dtype": dtype}
    if op in ("layer_norm", "layer_norm_vjp"):
        case = {"op": op, "rows": tokens(), "cols": size(64, 8192), "dtype": dtype, "weight": rng.choice([dtype, "f32"])}
        if op == "layer_norm":
            case["save"] = rng.random() < 0.5
        return case
    return {"op": op, "rows": rng.choice([size(1, 64), size(64, 1024)]), "vocab": size(512, 131072),
            "k": rng.choice([1, 8, 20, 64, 100, 256]), "dtype": dtype, "teacher": rng.choice([dtype, "f32"]),
            "tau": rng.choice([0.5, 1.0, 2.0]), "grad": rng.random() < 0.6}


def blocks(n):
    return (n + 127) // 128


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def activations(rows, cols):
        # a few channels of activations are many times larger than the others
        return normal(rows, cols) * torch.where(uniform(cols) < 0.01, 8.0, 1.0)

    s = dict(case)
    op = case["op"]
    if op == "blocks":
        R, C = case["rows"], case["cols"]
        x = activations(R, C) if case["block_rows"] == 1 else normal(R, C).mul_(1 / math.sqrt(C))
        s["x"] = x.to(DTYPES[case["dtype"]])
        return s
    if op == "linear_fp8":
        M, N, K = case["M"], case["N"], case["K"]

        def codes(r, c):
            # what quantization leaves: the largest of a block near 448
            return normal(r, c).mul_(150.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["a"], s["w"] = codes(M, K), codes(N, K)
        # a token's scales beside each other block by block, as the quantization lays them out
        s["a_scale"] = (uniform(blocks(K), M) * 0.01 + 0.002).t()
        s["w_scale"] = (uniform(blocks(N), blocks(K)) * 0.01 + 0.002) / math.sqrt(K)
        return s
    if op in ("layer_norm", "layer_norm_vjp"):
        R, C = case["rows"], case["cols"]
        x = activations(R, C) + normal(R, 1) * 0.3
        s["x"] = x.to(DTYPES[case["dtype"]])
        wt = DTYPES[case["weight"]]
        s["weight"] = (1 + 0.1 * normal(C)).to(wt)
        s["bias"] = (0.1 * normal(C)).to(wt)
        if op == "layer_norm_vjp":
            # what the forward pass saved, and the gradient that comes back to it
            v = s["x"].double()
            mean = v.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = (1 / torch.sqrt((v - mean[:, None]).square().mean(1) + EPS)).float()
            s["grad_y"] = (normal(R, C) * 0.1).to(DTYPES[case["dtype"]])
        return s
    R, V, k = case["rows"], case["vocab"], case["k"]
    logits = normal(R, V) * 2.0
    # the teacher's top entries, distinct tokens anywhere in the vocabulary, best first
    first = torch.randint(0, V, (R, 1), generator=g, device="cuda")
    step = torch.randint(1, max(2, V // k), (R, 1), generator=g, device="cuda")
    index = (first + step * torch.arange(k, device="cuda")) % V
    teacher = 12.0 - 1.5 * torch.arange(k, device="cuda").float().sqrt() + 0.2 * normal(R, k)
    logits.scatter_(1, index, teacher + 0.5 * normal(R, k))
    # some tokens carry no loss (a prompt, a padded sequence), some list fewer entries
    none = uniform(R, 1) < 0.1
    short = torch.where(uniform(R, 1) < 0.2, uniform(R, 1) * k, 1.0 * k)
    s["index"] = torch.where(none | (torch.arange(k, device="cuda") >= short.ceil()), -1, index)
    s["teacher"] = teacher.to(DTYPES[case["teacher"]])
    s["logits"] = logits.to(DTYPES[case["dtype"]])
    s["grad_loss"] = torch.where(none[:, 0], 0.0, (0.5 + uniform(R)))
    return s


# ---- plain forms ------------------------------------------------------------------------------

def plain_e4m3(v):
    """The nearest e4m3 values to 64-bit ones of magnitude up to 448, halves to even."""
    m, _ = torch.frexp(v)                              # v / m is a power of two above |v|, 16 steps
    step = torch.where(v == 0, 0.0, v / m / 16).clamp(min=2.0 ** -9)
    return (torch.round(v / step) * step).clamp(-448, 448).to(torch.float8_e4m3fn)


def plain_blocks(x, block_rows):
    R, C = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -C % 128, 0, -R % block_rows))
    t = x.unflatten(1, (-1, 128)).unflatten(0, (-1, block_rows))       # [R / br][br][C / 128][128]
    # the quotients decide at half steps: 64 bits
    scale = (t.abs().amax((1, 3)).double() / 448.0).float()
    s = scale.double()[:, None, :, None]
    q = plain_e4m3(torch.where(s > 0, t.double() / s, 0.0))
    return q.flatten(2).flatten(0, 1)[:R, :C], scale


def plain_linear_fp8(a, a_scale, w, w_scale, dt):
    K, N = a.shape[1], w.shape[0]
    sa = a_scale.repeat_interleave(128, 1)[:, :K]
    sw = w_scale.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return ((a.float() * sa) @ (w.float() * sw).t()).to(dt)


def plain_layer_norm(x, weight, bias):
    v = x.float()
    mean = v.mean(1)
    d = v - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
    return (d * rstd[:, None] * weight.float() + bias.float()).to(x.dtype), mean, rstd


def plain_layer_norm_vjp(x, weight, mean, rstd, grad_y):
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    g = grad_y.float()
    gw = g * weight.float()
    dx = rstd[:, None] * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
    return dx.to(x.dtype), (g * xh).sum(0).to(weight.dtype), g.sum(0).to(weight.dtype)


def plain_distill(logits, index, teacher, grad_loss, tau, grad):
    z, t = logits.float() / tau, teacher.float() / tau
    z = z - z.amax(1, keepdim=True)
    log_z = torch.log(torch.exp(z).sum(1, keepdim=True))
    there = index >= 0
    at = index.clamp(min=0)
    t = torch.where(there, t, -1e30)
    t = t - t.amax(1, keepdim=True)
    e = torch.where(there, torch.exp(t), 0.0)
    total = e.sum(1, keepdim=True)
    p = e / total.clamp(min=1e-30)
    log_p = t - torch.log(total.clamp(min=1e-30))
    loss = torch.where(there, p * (log_p - (z.gather(1, at) - log_z)), 0.0).sum(1)
    if not grad:
        return loss
    d = torch.exp(z - log_z) * there.any(1, keepdim=True)
    d.scatter_add_(1, at, -p)
    return loss, (d * (grad_loss / tau)[:, None]).to(logits.dtype)


def run(s):
    op = s["op"]
    if own:
        from trellis_coded_weight_amd import api
        if op == "blocks":
            return api.quantize_blocks(s["x"], block_rows=s["block_rows"])
        if op == "linear_fp8":
            return api.matmul_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"], dtype=DTYPES[s["dtype"]])
        if op == "layer_norm":
            return api.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, save=s["save"])
        if op == "layer_norm_vjp":
            return api.layer_norm_vjp(s["x"], s["weight"], s["mean"], s["rstd"], s["grad_y"])
        return api.distill_topk(s["logits"], s["index"], s["teacher"], temperature=s["tau"],
                                grad_loss=s["grad_loss"] if s["grad"] else None)
    if op == "blocks":
        return plain_blocks(s["x"], s["block_rows"])
    if op == "linear_fp8":
        return plain_linear_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"], DTYPES[s["dtype"]])
    if op == "layer_norm":
        y, mean, rstd = plain_layer_norm(s["x"], s["weight"], s["bias"])
        return (y, mean, rstd) if s["save"] else y
    if op == "layer_norm_vjp":
        return plain_layer_norm_vjp(s["x"], s["weight"], s["mean"], s["rstd"], s["grad_y"])
    return plain_distill(s["logits"], s["index"], s["teacher"], s["grad_loss"], s["tau"], s["grad"])


def work(case):
    op = case["op"]
    if op == "blocks":
        R, C = case["rows"], case["cols"]
        scales = blocks(R) * blocks(C) if case["block_rows"] == 128 else R * blocks(C)
        return {"bytes": R * C * (BYTES[case["dtype"]] + 1) + 4 * scales, "flops": 3 * R * C}
    if op == "linear_fp8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K + 4 * (M + blocks(N)) * blocks(K) + M * N * BYTES[case["dtype"]], "flops": 2 * M * N * K}
    if op in ("layer_norm", "layer_norm_vjp"):
        n, b, w = case["rows"] * case["cols"], BYTES[case["dtype"]], BYTES[case["weight"]]
        if op == "layer_norm":
            return {"bytes": 2 * n * b + 2 * case["cols"] * w + (8 * case["rows"] if case["save"] else 0), "flops": 7 * n}
        return {"bytes": 3 * n * b + 3 * case["cols"] * w + 8 * case["rows"], "flops": 14 * n}
    n = case["rows"] * case["vocab"]
    entries = case["rows"] * case["k"] * (8 + BYTES[case["teacher"]])
    # the logits in and, in training, their gradient out
    return {"bytes": n * BYTES[case["dtype"]] * (2 if case["grad"] else 1) + entries + 8 * case["rows"],
            "flops": n * (8 if case["grad"] else 4)}


# ---- the same from the definitions, in 64 bits -------------------------------------------------

def exact_values():
    """The 256 values of e4m3, from its bits: a sign, 4 of exponent (bias 7), 3 of mantissa; all
    ones is NaN."""
    out = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out.append(-v if b >> 7 else v)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def exact_rounded(v):
    """The e4m3 values nearest to |v| <= 448: the two neighbours in the list of them, and the even
    one where both are as near."""
    points = exact_values()[:127]                          # ascending, index = bits
    a = v.abs().clamp(max=448.0)
    hi = torch.searchsorted(points, a.contiguous()).clamp(1, 126)
    down, up = a - points[hi - 1], points[hi] - a
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    return torch.copysign(points[pick], v)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "blocks":
        R, C, br = case["rows"], case["cols"], case["block_rows"]
        q = torch.empty(R, C, dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.empty(-(-R // br), blocks(C), device="cuda")
        for j in range(blocks(C)):                         # a column of blocks at a time
            x = s["x"][:, 128 * j:128 * j + 128].double()
            largest = x.abs().max(1).values
            of_row = torch.arange(R, device="cuda") // br
            top = torch.zeros(scale.shape[0], dtype=torch.float64, device="cuda").scatter_reduce(0, of_row, largest, "amax")
            scale[:, j] = top / 448
            step = scale[:, j].double()[of_row].unsqueeze(1)
            q[:, 128 * j:128 * j + 128] = exact_rounded(torch.where(step == 0, 0.0, x / step)).float().to(q.dtype)
        return q, scale
    if op == "linear_fp8":
        values = exact_values()
        acc = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for j in range(blocks(case["K"])):
            a, w = (values[t[:, 128 * j:128 * j + 128].contiguous().view(torch.uint8).long()] for t in (s["a"], s["w"]))
            column = s["w_scale"][torch.arange(case["N"], device="cuda") // 128, j].double()
            acc += torch.mm(a * s["a_scale"][:, j:j + 1].double(), (w * column.unsqueeze(1)).t().contiguous())
        return acc
    if op == "layer_norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS).rsqrt()
        y = torch.addcmul(s["bias"].double(), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), s["weight"].double())
        return (y, mean, rstd) if case["save"] else y
    if op == "layer_norm_vjp":
        x, dy, w = s["x"].double(), s["grad_y"].double(), s["weight"].double()
        mean, rstd, n = s["mean"].double().unsqueeze(1), s["rstd"].double().unsqueeze(1), case["cols"]
        c = x - mean
        # d/dx of sum(dy w c rstd): through c, through the mean and through rstd
        dc = dy * w * rstd
        along = torch.sum(dy * w * c, 1, keepdim=True)
        dx = dc - dc.sum(1, keepdim=True) / n - c * rstd ** 3 * along / n
        return dx, torch.sum(dy * c * rstd, 0), torch.sum(dy, 0)
    tau = case["tau"]
    z = s["logits"].double().div_(tau)
    log_q = z.sub_(torch.logsumexp(z, 1, keepdim=True))
    masked = s["teacher"].double().div(tau).masked_fill(s["index"] < 0, -math.inf)
    empty = (s["index"] < 0).all(1)
    log_p = torch.where(empty.unsqueeze(1), -math.inf, torch.log_softmax(masked, 1))
    p = log_p.exp()
    row = torch.arange(case["rows"], device="cuda").unsqueeze(1)
    picked = log_q[row, s["index"].remainder(case["vocab"])]
    terms = p * (log_p.masked_fill(p == 0, 0.0) - picked)
    loss = terms.sum(1)
    if not case["grad"]:
        return loss
    q = log_q.exp_()
    q[empty] = 0
    q.index_put_((row.expand_as(p), s["index"].remainder(case["vocab"])), -p, accumulate=True)
    return loss, q.mul_((s["grad_loss"].double() / tau).unsqueeze(1))
