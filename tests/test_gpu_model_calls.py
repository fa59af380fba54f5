"""How the model operators are called: refusals, workspaces, streams, graphs, repeated calls, and
a run of them together as a model on coded weights uses them."""
import numpy as np
import pytest

import model_ref as ref
import test_gpu_blocks
import test_gpu_distill
from helpers import say
from test_gpu_graphs import capture
from test_gpu_layer_norm import normal
from test_gpu_matvec import random_words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    import torch
    assert torch.cuda.is_available(), "GPU test without a GPU"
    from trellis_coded_weight_amd import api as a
    return a


def refused(calls):
    import torch
    from trellis_coded_weight_amd._native import QtcqError
    say("model operators: refusals")
    for i, f in enumerate(calls):
        with pytest.raises((ValueError, QtcqError)):
            f()
            pytest.fail("call %d was taken" % i, pytrace=False)
    torch.cuda.synchronize()


def test_refusals_blocks(api):
    import torch
    x = normal(6, 300, dtype="bfloat16")
    q, s = api.quantize_blocks(x)
    w, ws = api.quantize_blocks(normal(40, 300, seed=2), block_rows=128)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    a100, s100 = api.quantize_blocks(normal(100, 300, seed=3))
    refused([lambda: api.quantize_blocks(x, block_rows=64), lambda: api.quantize_blocks(x.cpu()),
             lambda: api.quantize_blocks(x[0]), lambda: api.quantize_blocks(x.t()), lambda: api.quantize_blocks(x.int()),
             lambda: api.quantize_blocks(x.as_strided((6, 300), (299, 1))), lambda: api.quantize_blocks(q),
             lambda: api.matmul_fp8(q, s, w, ws, dtype=torch.int8), lambda: api.matmul_fp8(x, s, w, ws),
             lambda: api.matmul_fp8(q, s, w[:, :299], ws), lambda: api.matmul_fp8(q, s[:5], w, ws),
             lambda: api.matmul_fp8(q, s[:, :2], w, ws), lambda: api.matmul_fp8(q, s, w, s),
             lambda: api.matmul_fp8(q, s.double(), w, ws), lambda: api.matmul_fp8(q, s, w, ws.cpu()),
             lambda: api.matmul_fp8(q.view(torch.uint8), s, w, ws), lambda: api.matmul_fp8(q, s, w.t(), ws),
             lambda: api.matmul_fp8(a100[:, :299], s100, w[:, :299], ws, workspace=small),
             lambda: api.matmul_fp8(a100[:, :299], s100, w[:, :299], ws, workspace=small.cpu())])


def test_refusals_layer_norm(api):
    import torch
    x, gy = normal(1700, 64, dtype="float16"), normal(1700, 64, seed=2, dtype="float16")
    w, b = normal(64, seed=3), normal(64, seed=4)
    y, mean, rstd = api.layer_norm(x, w, b, save=True)
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    grad = w.clone().requires_grad_()
    refused([lambda: api.layer_norm(x, w.half(), b), lambda: api.layer_norm(x, w.bfloat16(), b.bfloat16()),
             lambda: api.layer_norm(x, w[:63], b), lambda: api.layer_norm(x, w, b[:1]), lambda: api.layer_norm(x, w, b, eps=-1.0),
             lambda: api.layer_norm(x, w, b, eps=float("nan")), lambda: api.layer_norm(x.cpu(), w, b),
             lambda: api.layer_norm(x, w.cpu(), b), lambda: api.layer_norm(x, normal(128)[::2], b),
             lambda: api.layer_norm(x, grad, b), lambda: api.layer_norm(x.double(), w, b), lambda: api.layer_norm(x[0], w, b),
             lambda: api.layer_norm_vjp(x, w, mean, rstd, gy.float()), lambda: api.layer_norm_vjp(x, w, mean, rstd, gy[:5]),
             lambda: api.layer_norm_vjp(x, w, mean[:4], rstd, gy), lambda: api.layer_norm_vjp(x, w, mean, None, gy),
             lambda: api.layer_norm_vjp(x, w, mean, rstd.half(), gy), lambda: api.layer_norm_vjp(x, w[:5], mean, rstd, gy),
             lambda: api.layer_norm_vjp(x, w, mean, rstd, gy, workspace=small)])
    with torch.no_grad():
        assert torch.equal(api.layer_norm(x, grad, b), api.layer_norm(x, grad.detach(), b))
    assert api.layer_norm_vjp(x, w, mean, rstd, gy, want_x=False, want_w=False) == (None, None, None)


def test_refusals_distill(api):
    import torch
    z, index, t, gl = test_gpu_distill.inputs(4, 70000, 8, "bfloat16")
    loss, stats = api.distill_topk(z, index, t, save=True)
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    many = torch.zeros(4, 1025, dtype=torch.int64, device="cuda")
    refused([lambda: api.distill_topk(z, index, t, temperature=0.0), lambda: api.distill_topk(z, index, t, temperature=-1.0),
             lambda: api.distill_topk(z, index, t, temperature=float("nan")),
             lambda: api.distill_topk(z, index, t, temperature=2.0 ** 101),
             lambda: api.distill_topk(z, index[:3], t[:3]), lambda: api.distill_topk(z, index, t[:, :7]),
             lambda: api.distill_topk(z, index.short(), t), lambda: api.distill_topk(z, index.float(), t),
             lambda: api.distill_topk(z, index, t.double()), lambda: api.distill_topk(z.cpu(), index, t),
             lambda: api.distill_topk(z, index.cpu(), t), lambda: api.distill_topk(z, index, t, grad_loss=gl[:3]),
             lambda: api.distill_topk(z, index, t, grad_loss=gl.half()), lambda: api.distill_topk(z, index, t, grad_loss=gl, save=True),
             lambda: api.distill_topk(z, index, t, teacher_log_z=3.0), lambda: api.distill_topk(z, index, t, grad_loss=1.0),
             lambda: api.distill_topk(z, index, t, teacher_log_z=gl[:1]), lambda: api.distill_topk(z, index, t, workspace=small),
             lambda: api.distill_topk(z.float().requires_grad_(), index, t),
             lambda: api.distill_topk(z, many, many.float()),
             lambda: api.distill_topk_vjp(z, index, t, stats[:, :4], gl), lambda: api.distill_topk_vjp(z, index, t, stats.half(), gl),
             lambda: api.distill_topk_vjp(z, index, t, stats[:3], gl), lambda: api.distill_topk_vjp(z, index, t, None, gl),
             lambda: api.distill_topk_vjp(z, index, t, stats, None), lambda: api.distill_topk_vjp(z, index, t, stats, gl[:2]),
             lambda: api.distill_topk_vjp(z, index, t, stats, gl, temperature=0.0)])


def every_call(api, seed=0, scale=1.0):
    """(function without arguments, the tensors it reads) for each operator, in several of its
    kernels; workspaces are the callers', and hold garbage."""
    import torch
    calls = []

    def ws(n):
        return torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    for R, C, br in ((5, 700, 1), (300, 1000, 128)):
        x = normal(R, C, seed=seed + 1, dtype="bfloat16", scale=scale)
        calls.append((lambda x=x, br=br: api.quantize_blocks(x, block_rows=br), [x]))
    from trellis_coded_weight_amd import _native as nat
    for M, N, K in ((7, 300, 512), (70, 400, 4112), (70, 400, 4099), (600, 700, 640)):
        o = test_gpu_blocks.operands(M, N, K)
        o[1].mul_(scale)
        w = ws(nat.qtcq_matmul_fp8_workspace_bytes(M, N, K, K % 16 == 0))
        calls.append((lambda o=o, w=w: api.matmul_fp8(*o, dtype=torch.bfloat16, workspace=w), [o[1]]))
    for R, C in ((9, 1000), (1700, 1000), (5, 20000)):
        x, gy = normal(R, C, seed=seed + 2, scale=scale), normal(R, C, seed=seed + 3)
        w, b = normal(C, seed=4), normal(C, seed=5)
        g = ws(nat.qtcq_layer_norm_vjp_workspace_bytes(R, C))

        def norm(x=x, gy=gy, w=w, b=b, g=g):
            y, mean, rstd = api.layer_norm(x, w, b, save=True)
            return (y, mean, rstd) + api.layer_norm_vjp(x, w, mean, rstd, gy, workspace=g)
        calls.append((norm, [x]))
    for R, V, k in ((4, 900, 5), (700, 5000, 20), (3, 70001, 64)):
        z, index, t, gl = test_gpu_distill.inputs(R, V, k, "float32", seed=seed)
        z.mul_(scale)
        d = ws(nat.qtcq_distill_topk_workspace_bytes(R, V))

        def distill(z=z, index=index, t=t, gl=gl, d=d):
            loss, grad = api.distill_topk(z, index, t, grad_loss=gl, workspace=d)
            saved, stats = api.distill_topk(z, index, t, save=True, workspace=d)
            return loss, grad, saved, stats, api.distill_topk_vjp(z, index, t, stats, gl)
        calls.append((distill, [z]))
    return calls


def flat(out):
    return [out] if not isinstance(out, (tuple, list)) else list(out)


def same(a, b):
    import torch
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}
    return all(torch.equal(x.view(bits[x.element_size()]), y.view(bits[y.element_size()]))
               for x, y in zip(flat(a), flat(b)))


def test_repeated_calls_give_the_same_bits(api):
    import torch
    say("model operators: repeated calls")
    for f, _ in every_call(api):
        first = f()
        for _ in range(3):
            assert same(first, f())
    torch.cuda.synchronize()


def test_two_streams_at_once(api):
    """Calls of both streams interleaved, each with inputs, outputs and workspaces of its own."""
    import torch
    say("model operators: two streams")
    one, two = every_call(api, 1), every_call(api, 2, 0.5)
    want = [[f() for f, _ in calls] for calls in (one, two)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        got = [[], []]
        for (f, _), (g, _) in zip(one, reversed(two)):
            with torch.cuda.stream(streams[0]):
                got[0].append(f())
            with torch.cuda.stream(streams[1]):
                got[1].append(g())
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got[0], want[0]))
    assert all(same(a, b) for a, b in zip(reversed(got[1]), want[1]))


def test_captured_and_replayed(api):
    """All of them in one graph; each replay, with other inputs, against the eager calls."""
    import torch
    say("model operators: graph")
    calls = every_call(api)
    g, out = capture(lambda: [f() for f, _ in calls])
    for rep in range(3):
        for _, inputs in calls:
            for x in inputs:
                x.mul_(0.75)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        eager = [f() for f, _ in calls]
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, eager)):
            assert same(a, b), (rep, i)


def test_two_graphs_with_workspaces_of_their_own(api):
    """Graphs captured without given workspaces keep what they allocate."""
    import torch
    z, index, t, gl = test_gpu_distill.inputs(3, 70001, 20, "bfloat16")
    o = test_gpu_blocks.operands(70, 400, 4099)
    say("model operators: two graphs")
    f = lambda: [*api.distill_topk(z, index, t, grad_loss=gl), api.matmul_fp8(*o)]      # noqa: E731
    want = f()
    (g1, a), (g2, b) = capture(f), capture(f)
    for _ in range(3):
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert same(a, want) and same(b, want)


def coded(api, M, N, seed):
    import torch
    words = torch.from_numpy(random_words(M, N, 16, False, seed).view(np.int32)).cuda()
    return api.decode_matrix(words, M, N, dtype=torch.bfloat16)


class Student:
    """One block of a model on coded weights, and its distillation from a teacher's top logits:
    layer norm, a projection and the head in e4m3; back through the head and the projection
    with the decoded weights to the norm's gradients."""

    def __init__(self, api, tokens, width, hidden, vocab):
        self.api = api
        self.w1, self.head = coded(api, hidden, width, 5), coded(api, vocab, hidden, 6)
        self.q1, self.qh = (api.quantize_blocks(w, block_rows=128) for w in (self.w1, self.head))
        self.x = normal(tokens, width, seed=7, dtype="bfloat16", scale=2.0)
        self.weight, self.bias = normal(width, seed=8) * 0.2 + 1, normal(width, seed=9) * 0.1
        _, self.index, self.teacher, self.grad_loss = test_gpu_distill.inputs(tokens, vocab, 16, "float32", seed=10)

    def step(self):
        import torch
        api, bf16 = self.api, torch.bfloat16
        y, mean, rstd = api.layer_norm(self.x, self.weight, self.bias, save=True)
        a, sa = api.quantize_blocks(y)
        h = api.matmul_fp8(a, sa, *self.q1, dtype=bf16)
        b, sb = api.quantize_blocks(h)
        z = api.matmul_fp8(b, sb, *self.qh, dtype=bf16)
        loss, gz = api.distill_topk(z, self.index, self.teacher, temperature=2.0, grad_loss=self.grad_loss)
        gy = (gz @ self.head) @ self.w1
        return (y, mean, rstd, a, sa, h, b, sb, z, loss, gz, gy) + api.layer_norm_vjp(self.x, self.weight, mean, rstd, gy)


@pytest.mark.parametrize("tokens,width,hidden,vocab", [(1, 512, 256, 1024), (37, 512, 304, 2000), (300, 1024, 640, 4096)])
def test_a_run_of_them_together(api, tokens, width, hidden, vocab):
    """Each result against 64 bits on what the ones before it gave, and the losses against the
    whole chain in 64 bits with the decoded weights as they are."""
    import torch
    s = Student(api, tokens, width, hidden, vocab)
    say("model operators together %dx%dx%dx%d" % (tokens, width, hidden, vocab))
    out = s.step()
    torch.cuda.synchronize()
    y, mean, rstd, a, sa, h, b, sb, z, loss, gz, gy, gx, gw, gb = out
    want, e, m, em, r, er = ref.layer_norm(s.x, s.weight.double(), s.bias.double(), 1e-5)
    for got, v, bound in ((y, want, e), (mean, m, em), (rstd, r, er)):
        ref.within(got, v, bound, "norm")
    for x, q, scale, br in ((y, a, sa, 1), (h, b, sb, 1), (s.w1, *s.q1, 128), (s.head, *s.qh, 128)):
        bits, v = ref.quantize_blocks(x, br)
        assert torch.equal(q.view(torch.uint8), bits) and torch.equal(scale, v)
    ref.within(h, *ref.matmul_fp8(a, sa, *s.q1, torch.bfloat16), "projection")
    ref.within(z, *ref.matmul_fp8(b, sb, *s.qh, torch.bfloat16), "head")
    v, e, g, eg = ref.distill(z, s.index, s.teacher, 2.0, None, s.grad_loss, z.dtype)
    ref.within(loss, v, e, "loss")
    ref.within(gz, g, eg, "gradient of the logits")
    for got, (v, e) in zip((gx, gw, gb), ref.layer_norm_vjp(s.x, s.weight.double(), mean, rstd, gy, torch.float32)):
        ref.within(got, v, e, "gradients of the norm")


def test_a_run_of_them_in_a_graph(api):
    import torch
    s = Student(api, 48, 512, 304, 2000)
    say("model operators together in a graph")
    g, out = capture(s.step)
    for rep in range(3):
        s.x.copy_(normal(48, 512, seed=20 + rep, dtype="bfloat16"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        eager = s.step()
        torch.cuda.synchronize()
        assert same(out, eager), rep
