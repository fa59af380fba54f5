"""The dense operators' C entry points refuse bad arguments before launching anything, and
their size query gives the documented sizes.  No GPU needed."""
import pytest

FAKE = 1 << 20   # a non-NULL, aligned pointer value; never dereferenced by validation paths


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


def test_quantize_rows(nat):
    call = caller(nat, "qtcq_quantize_rows", ["x", "dtype", "rows", "cols", "ldx", "q", "ldq", "scale", "stream"],
                  [FAKE, nat.QTCQ_BF16, 4, 64, 64, FAKE, 64, FAKE, None])
    bad, no = nat.QTCQ_ERR_INVALID_ARG, nat.QTCQ_ERR_UNSUPPORTED
    for kw in (dict(rows=-1), dict(cols=-1), dict(ldx=63), dict(ldq=63), dict(x=None), dict(q=None),
               dict(scale=None), dict(x=FAKE + 1), dict(scale=FAKE + 2), dict(dtype=nat.QTCQ_F32, x=FAKE + 2)):
        assert call(**kw) == bad, kw
    for kw in (dict(dtype=nat.QTCQ_I8), dict(dtype=7), dict(dtype=-1), dict(rows=(1 << 24) + 1),
               dict(cols=(1 << 24) + 1, ldx=1 << 25, ldq=1 << 25)):
        assert call(**kw) == no, kw
    assert call(rows=0, x=None, q=None, scale=None) == nat.QTCQ_OK


def test_decode_matrix(nat):
    call = caller(nat, "qtcq_decode_matrix",
                  ["bits", "M", "N", "L", "k", "code", "tb", "dtype", "w", "ldw", "scale", "stream"],
                  [FAKE, 32, 64, 16, 2, 0, 0, nat.QTCQ_I8, FAKE, 64, FAKE, None])
    bad, no = nat.QTCQ_ERR_INVALID_ARG, nat.QTCQ_ERR_UNSUPPORTED
    for kw in (dict(M=-16), dict(N=-16), dict(M=8), dict(N=40), dict(ldw=48), dict(ldw=72), dict(bits=None),
               dict(w=None), dict(scale=None), dict(w=FAKE + 8), dict(scale=FAKE + 1), dict(bits=FAKE + 2),
               dict(dtype=nat.QTCQ_BF16, ldw=68), dict(dtype=nat.QTCQ_F32, ldw=66)):
        assert call(**kw) == bad, kw
    for kw in (dict(L=7), dict(L=18), dict(k=3), dict(code=3), dict(dtype=4), dict(dtype=-1),
               dict(M=(1 << 24) + 16)):
        assert call(**kw) == no, kw
    assert call(M=0, bits=None, w=None, scale=None) == nat.QTCQ_OK
    assert call(N=0, dtype=nat.QTCQ_F16, bits=None, w=None, scale=None) == nat.QTCQ_OK


def test_matmul_int8(nat):
    call = caller(nat, "qtcq_matmul_int8",
                  ["a", "lda", "sa", "w", "ldw", "sw", "M", "N", "K", "dtype", "y", "ldy", "ws", "wsb",
                   "stream"],
                  [FAKE, 64, FAKE, FAKE, 64, FAKE, 4, 8, 64, nat.QTCQ_F32, FAKE, 8, None, 0, None])
    bad, no = nat.QTCQ_ERR_INVALID_ARG, nat.QTCQ_ERR_UNSUPPORTED
    for kw in (dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=63), dict(ldw=63), dict(ldy=7), dict(a=None),
               dict(w=None), dict(sa=None), dict(sw=None), dict(y=None), dict(y=FAKE + 2), dict(sa=FAKE + 2),
               dict(sw=FAKE + 1), dict(dtype=nat.QTCQ_F16, y=FAKE + 1)):
        assert call(**kw) == bad, kw
    big = 1 << 25
    for kw in (dict(dtype=nat.QTCQ_I8), dict(dtype=9), dict(K=131072, lda=big, ldw=big), dict(M=(1 << 24) + 1),
               dict(N=(1 << 24) + 1, ldy=big), dict(M=1 << 24, N=1 << 24, ldy=big)):
        assert call(**kw) == no, kw
    assert call(M=0, a=None, sa=None, y=None) == nat.QTCQ_OK
    assert call(N=0, w=None, sw=None, y=None) == nat.QTCQ_OK
    # a result of one tile and a long sum: shares of k; rows of 65 bytes: copies too
    size = nat.qtcq_matmul_int8_workspace_bytes
    ws = size(100, 256, 65536, True)
    assert ws >= 2 * 100 * 256 * 4 and size(100, 256, 65536, False) > ws
    assert size(1, 256, 65536, True) == 0 and size(4096, 4096, 4096, True) == 0
    assert size(-1, 8, 8, True) == 0 and size(8, 8, 131072, True) == 0
    wide = dict(M=100, N=256, K=65536, lda=65536, ldw=65536, ldy=256)
    for kw in (dict(ws=None, wsb=ws), dict(ws=FAKE + 8, wsb=ws), dict(ws=FAKE, wsb=ws - 1),
               dict(ws=FAKE, wsb=ws, ldw=65537), dict(ws=FAKE, wsb=ws, a=FAKE + 1)):
        assert call(**dict(wide, **kw)) == nat.QTCQ_ERR_WORKSPACE, kw


def test_gated_forward(nat):
    call = caller(nat, "qtcq_gated_forward",
                  ["x", "ldx", "wg", "wu", "ldw", "dtype", "M", "F", "K", "act", "h", "ldh", "gate", "up", "ldg",
                   "ws", "wsb", "stream"],
                  [FAKE, 64, FAKE, FAKE, 64, nat.QTCQ_BF16, 4, 8, 64, 0, FAKE, 8, FAKE, FAKE, 8, None, 0, None])
    bad, no = nat.QTCQ_ERR_INVALID_ARG, nat.QTCQ_ERR_UNSUPPORTED
    for kw in (dict(M=-1), dict(F=-1), dict(K=-1), dict(ldx=63), dict(ldw=63), dict(ldh=7), dict(ldg=7),
               dict(gate=None), dict(up=None), dict(x=None), dict(wg=None), dict(wu=None), dict(h=None),
               dict(x=FAKE + 1), dict(wg=FAKE + 1), dict(wu=FAKE + 1), dict(h=FAKE + 1), dict(gate=FAKE + 1),
               dict(up=FAKE + 1)):
        assert call(**kw) == bad, kw
    big = 1 << 25
    for kw in (dict(dtype=nat.QTCQ_F32), dict(dtype=nat.QTCQ_I8), dict(dtype=5), dict(act=-1), dict(act=5),
               dict(M=(1 << 24) + 1), dict(K=(1 << 21) + 1, ldx=big, ldw=big),
               dict(M=1 << 24, F=1 << 21, ldh=big, ldg=big)):
        assert call(**kw) == no, kw
    assert call(M=0, x=None, h=None) == nat.QTCQ_OK
    assert call(F=0, wg=None, wu=None, h=None) == nat.QTCQ_OK
    size = nat.qtcq_gated_workspace_bytes
    ws = size(100, 128, 32768, True)
    assert ws >= 2 * 2 * 100 * 128 * 4 and size(100, 128, 32768, False) > ws
    assert size(1, 128, 32768, True) == 0 and size(8, 8, (1 << 21) + 1, True) == 0
    wide = dict(M=100, F=128, K=32768, ldx=32768, ldw=32768, ldh=128, ldg=128)
    for kw in (dict(ws=None, wsb=ws), dict(ws=FAKE + 8, wsb=ws), dict(ws=FAKE, wsb=ws - 1),
               dict(ws=FAKE, wsb=ws, ldx=32769), dict(ws=FAKE, wsb=ws, wu=FAKE + 2)):
        assert call(**dict(wide, **kw)) == nat.QTCQ_ERR_WORKSPACE, kw


def test_gated_vjp(nat):
    size = nat.qtcq_gated_vjp_workspace_bytes
    ws = size(4, 8, 64, True)
    assert ws >= 2 * 2 * 4 * 8 and ws % 256 == 0
    assert size(4, 8, 64, False) > ws
    assert size(-1, 8, 64, True) == 0
    assert size(4, (1 << 21) + 1, 64, True) == 0
    assert size(1 << 20, 1 << 20, 64, True) == 0
    call = caller(nat, "qtcq_gated_vjp",
                  ["x", "ldx", "wg", "wu", "ldw", "gate", "up", "ldg", "gh", "ldgh", "dtype", "M", "F", "K", "act",
                   "gx", "ldgx", "gwg", "gwu", "ldgw", "ws", "wsb", "stream"],
                  [FAKE, 64, FAKE, FAKE, 64, FAKE, FAKE, 8, FAKE, 8, nat.QTCQ_F16, 4, 8, 64, 0, FAKE, 64, FAKE, FAKE,
                   64, FAKE, ws, None])
    bad, no, small = nat.QTCQ_ERR_INVALID_ARG, nat.QTCQ_ERR_UNSUPPORTED, nat.QTCQ_ERR_WORKSPACE
    for kw in (dict(M=-1), dict(F=-1), dict(K=-1), dict(ldx=63), dict(ldw=63), dict(ldg=7), dict(ldgh=7),
               dict(ldgx=63), dict(ldgw=63), dict(gwg=None), dict(gwu=None), dict(x=None), dict(wg=None),
               dict(wu=None), dict(gate=None), dict(up=None), dict(gh=None), dict(gx=FAKE + 1), dict(gwg=FAKE + 1),
               dict(gwu=FAKE + 1), dict(gh=FAKE + 1), dict(x=FAKE + 1)):
        assert call(**kw) == bad, kw
    for kw in (dict(dtype=nat.QTCQ_F32), dict(act=5), dict(M=(1 << 24) + 1)):
        assert call(**kw) == no, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(wsb=ws - 1)):
        assert call(**kw) == small, kw
    assert call(x=FAKE + 2) == small and call(ldw=65) == small
    assert call(gx=None, gwg=None, gwu=None) == nat.QTCQ_OK
    assert call(K=0) == nat.QTCQ_OK
    assert call(M=0, gwg=None, gwu=None) == nat.QTCQ_OK
