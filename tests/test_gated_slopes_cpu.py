"""The gated gradient's workspace holds its two slopes in two parts each, and only its own
entry point takes the request for rounded ones.  No GPU needed."""
import pytest

FAKE = 1 << 20   # a non-NULL, aligned pointer value; never dereferenced by validation paths


@pytest.fixture(scope="module")
def nat():
    from trellis_coded_weight_amd import _native
    return _native


@pytest.mark.parametrize("M,F,K", [(1, 64, 64), (120, 14336, 4096), (333, 2731, 1001)])
def test_workspace_holds_two_parts(nat, M, F, K):
    pitch = (F + 63) // 64 * 64
    for whole in (True, False):
        assert nat.qtcq_gated_vjp_workspace_bytes(M, F, K, whole) >= 2 * 2 * 2 * M * pitch


def test_request_for_rounded_slopes(nat):
    ws = nat.qtcq_gated_vjp_workspace_bytes(4, 8, 64, True)

    def vjp(act, wsb):
        return nat.raw_status("qtcq_gated_vjp", FAKE, 64, FAKE, FAKE, 64, FAKE, FAKE, 8, FAKE, 8, nat.QTCQ_F16, 4, 8, 64,
                              act, FAKE, 64, FAKE, FAKE, 64, FAKE, wsb, None)

    flag = nat.QTCQ_ACT_ROUND_SLOPES
    for act in (flag + 5, flag | 0x200, 0x200, -1, -flag, flag - 1):
        assert vjp(act, ws) == nat.QTCQ_ERR_UNSUPPORTED, act
    # one part of each takes half the scratch: refused below that
    assert vjp(nat.QTCQ_ACT_SILU, ws - 1) == nat.QTCQ_ERR_WORKSPACE
    assert vjp(nat.QTCQ_ACT_SILU | flag, ws // 2 - 1) == nat.QTCQ_ERR_WORKSPACE
    assert nat.raw_status("qtcq_gated_forward", FAKE, 64, FAKE, FAKE, 64, nat.QTCQ_F16, 4, 8, 64, flag, FAKE, 8, None,
                          None, 0, None, 0, None) == nat.QTCQ_ERR_UNSUPPORTED
