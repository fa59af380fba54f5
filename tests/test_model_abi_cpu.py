"""The model operators' C entry points refuse bad arguments before launching anything, and their
size queries give the documented sizes.  No GPU needed."""
import pytest

FAKE = 1 << 20   # a non-NULL, aligned pointer value; never dereferenced by validation paths
BIG = 1 << 25


@pytest.fixture(scope="module")
def nat():
    from trellis_coded_weight_amd import _native
    return _native


def caller(nat, name, names, ok):
    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[names.index(k)] = v
        return nat.raw_status(name, *a)
    return call


def refused(nat, call, bad, no):
    for kw in bad:
        assert call(**kw) == nat.QTCQ_ERR_INVALID_ARG, kw
    for kw in no:
        assert call(**kw) == nat.QTCQ_ERR_UNSUPPORTED, kw


def test_quantize_blocks(nat):
    call = caller(nat, "qtcq_quantize_blocks",
                  ["x", "dtype", "rows", "cols", "ldx", "br", "q", "ldq", "scale", "srow", "scol", "stream"],
                  [FAKE, nat.QTCQ_BF16, 4, 300, 300, 1, FAKE, 300, FAKE, 1, 4, None])
    refused(nat, call,
            (dict(rows=-1), dict(cols=-1), dict(ldx=299), dict(ldq=299), dict(x=None), dict(q=None), dict(scale=None),
             dict(x=FAKE + 1), dict(scale=FAKE + 2), dict(dtype=nat.QTCQ_F32, x=FAKE + 2), dict(srow=0), dict(scol=0),
             dict(scol=3), dict(srow=-1), dict(srow=2, scol=1), dict(srow=1, scol=1), dict(br=128, srow=1, scol=0)),
            (dict(dtype=nat.QTCQ_I8), dict(dtype=-1), dict(dtype=4), dict(br=0), dict(br=64), dict(br=-1),
             dict(rows=(1 << 24) + 1), dict(cols=(1 << 24) + 1, ldx=BIG, ldq=BIG),
             dict(rows=1 << 24, cols=1 << 17, ldx=BIG, ldq=BIG, scol=BIG)))
    assert call(rows=0, x=None, q=None, scale=None) == nat.QTCQ_OK
    assert call(cols=0, x=None, q=None, scale=None) == nat.QTCQ_OK


def test_matmul_fp8(nat):
    call = caller(nat, "qtcq_matmul_fp8",
                  ["a", "lda", "sa", "sar", "sac", "w", "ldw", "sw", "swr", "swc", "M", "N", "K", "dtype", "y", "ldy", "ws",
                   "wsb", "stream"],
                  [FAKE, 64, FAKE, 1, 4, FAKE, 64, FAKE, 1, 1, 4, 8, 64, nat.QTCQ_F32, FAKE, 8, None, 0, None])
    refused(nat, call,
            (dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=63), dict(ldw=63), dict(ldy=7), dict(a=None), dict(w=None),
             dict(sa=None), dict(sw=None), dict(y=None), dict(y=FAKE + 2), dict(sa=FAKE + 2), dict(sw=FAKE + 1),
             dict(dtype=nat.QTCQ_F16, y=FAKE + 1), dict(sar=-1), dict(sac=-1), dict(swr=-1), dict(swc=-4)),
            (dict(dtype=nat.QTCQ_I8), dict(dtype=9), dict(K=(1 << 22) + 1, lda=BIG, ldw=BIG), dict(M=(1 << 24) + 1),
             dict(N=(1 << 24) + 1, ldy=BIG), dict(M=1 << 24, N=1 << 24, ldy=BIG), dict(sar=(1 << 20) + 1)))
    assert call(M=0, a=None, sa=None, y=None) == nat.QTCQ_OK
    assert call(N=0, w=None, sw=None, y=None) == nat.QTCQ_OK
    size = nat.qtcq_matmul_fp8_workspace_bytes
    assert size(-1, 8, 8, True) == 0 and size(8, 8, (1 << 22) + 1, True) == 0


def test_layer_norm(nat):
    call = caller(nat, "qtcq_layer_norm",
                  ["x", "dtype", "rows", "cols", "ldx", "w", "b", "wdtype", "eps", "y", "ldy", "mean", "rstd", "stream"],
                  [FAKE, nat.QTCQ_BF16, 4, 64, 64, FAKE, FAKE, nat.QTCQ_F32, 1e-5, FAKE, 64, FAKE, FAKE, None])
    refused(nat, call,
            (dict(rows=-1), dict(cols=-1), dict(ldx=63), dict(ldy=63), dict(x=None), dict(y=None), dict(mean=None),
             dict(rstd=None), dict(eps=-1.0), dict(eps=float("nan")), dict(x=FAKE + 1), dict(y=FAKE + 1), dict(w=FAKE + 2),
             dict(b=FAKE + 1), dict(mean=FAKE + 2), dict(rstd=FAKE + 1)),
            (dict(dtype=nat.QTCQ_I8), dict(dtype=7), dict(wdtype=nat.QTCQ_F16), dict(dtype=nat.QTCQ_F32, wdtype=nat.QTCQ_BF16),
             dict(rows=(1 << 24) + 1), dict(cols=(1 << 24) + 1, ldx=BIG, ldy=BIG)))
    assert call(rows=0, x=None, y=None) == nat.QTCQ_OK
    assert call(cols=0, x=None, y=None) == nat.QTCQ_OK


def test_layer_norm_vjp(nat):
    size = nat.qtcq_layer_norm_vjp_workspace_bytes
    ws = size(2000, 64)
    assert ws >= 2 * 64 * 4 and size(1 << 20, 128) > ws and size(4, 64) == 0
    assert size(-1, 8) == 0 and size(8, -1) == 0 and size((1 << 24) + 1, 8) == 0
    call = caller(nat, "qtcq_layer_norm_vjp",
                  ["x", "dtype", "rows", "cols", "ldx", "w", "wdtype", "mean", "rstd", "gy", "ldgy", "gx", "ldgx", "gw",
                   "gb", "ws", "wsb", "stream"],
                  [FAKE, nat.QTCQ_F16, 2000, 64, 64, FAKE, nat.QTCQ_F16, FAKE, FAKE, FAKE, 64, FAKE, 64, FAKE, FAKE, FAKE, ws,
                   None])
    refused(nat, call,
            (dict(rows=-1), dict(cols=-1), dict(ldx=63), dict(ldgy=63), dict(ldgx=63), dict(x=None), dict(mean=None),
             dict(rstd=None), dict(gy=None), dict(x=FAKE + 1), dict(gy=FAKE + 1), dict(gx=FAKE + 1), dict(gw=FAKE + 1),
             dict(gb=FAKE + 1), dict(w=FAKE + 1), dict(mean=FAKE + 2)),
            (dict(dtype=nat.QTCQ_I8), dict(wdtype=nat.QTCQ_BF16), dict(rows=(1 << 24) + 1)))
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(wsb=ws - 1)):
        assert call(**kw) == nat.QTCQ_ERR_WORKSPACE, kw
    assert call(gx=None, gw=None, gb=None) == nat.QTCQ_OK
    assert call(cols=0, x=None) == nat.QTCQ_OK
    assert call(rows=0, gw=None, gb=None) == nat.QTCQ_OK


DISTILL = ["z", "dtype", "rows", "vocab", "ldl", "index", "ib", "ldi", "t", "tdtype", "ldt", "k", "tau"]
BAD = (dict(rows=-1), dict(vocab=-1), dict(k=-1), dict(ldl=99), dict(ldi=7), dict(ldt=7), dict(tau=0.0), dict(tau=-1.0),
       dict(tau=float("nan")), dict(z=None), dict(index=None), dict(t=None), dict(z=FAKE + 1), dict(index=FAKE + 4),
       dict(t=FAKE + 2), dict(ldg=99), dict(grad=FAKE + 1), dict(gl=None), dict(gl=FAKE + 2), dict(stats=FAKE + 2))
NO = (dict(dtype=3), dict(dtype=-1), dict(tdtype=3), dict(ib=2), dict(ib=16), dict(k=1025, ldi=2000, ldt=2000),
      dict(vocab=(1 << 24) + 1, ldl=BIG), dict(rows=(1 << 24) + 1), dict(tau=1e-31), dict(tau=1e31), dict(tau=float("inf")))


def test_distill_topk(nat):
    size = nat.qtcq_distill_topk_workspace_bytes
    ws = size(4, 100000)
    assert ws >= 4 * 5 * 4 and size(4, 100) == 0 and size(100000, 100000) == 0
    assert size(-1, 8) == 0 and size(8, -1) == 0 and size(8, (1 << 24) + 1) == 0
    call = caller(nat, "qtcq_distill_topk",
                  DISTILL + ["tlz", "loss", "stats", "gl", "grad", "ldg", "ws", "wsb", "stream"],
                  [FAKE, nat.QTCQ_BF16, 4, 100, 100, FAKE, 8, 8, FAKE, nat.QTCQ_F32, 8, 8, 1.0, None, FAKE, FAKE, FAKE, FAKE,
                   100, None, 0, None])
    refused(nat, call, BAD + (dict(loss=None), dict(loss=FAKE + 2), dict(tlz=FAKE + 1)), NO)
    wide = dict(vocab=100000, ldl=100000, ldg=100000)
    for kw in (dict(ws=None, wsb=ws), dict(ws=FAKE + 8, wsb=ws), dict(ws=FAKE, wsb=ws - 1)):
        assert call(**dict(wide, **kw)) == nat.QTCQ_ERR_WORKSPACE, kw
    assert call(rows=0, z=None, index=None, t=None, loss=None) == nat.QTCQ_OK


def test_distill_topk_vjp(nat):
    call = caller(nat, "qtcq_distill_topk_vjp", DISTILL + ["stats", "gl", "grad", "ldg", "stream"],
                  [FAKE, nat.QTCQ_BF16, 4, 100, 100, FAKE, 8, 8, FAKE, nat.QTCQ_F32, 8, 8, 1.0, FAKE, FAKE, FAKE, 100, None])
    refused(nat, call, BAD + (dict(stats=None), dict(grad=None)), NO)
    assert call(rows=0, z=None, index=None, t=None) == nat.QTCQ_OK
    assert call(vocab=0, z=None, grad=None) == nat.QTCQ_OK
