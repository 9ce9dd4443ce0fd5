"""Host side of the mixer operators, without a GPU: settings, sizes at the ends of
their types, the plan of a cut prompt, the build and the checks of the binding."""
import pytest
import torch

E, U = -1, -4


@pytest.fixture(scope="module")
def M():
    from bit_recurrent_state_decode_b200 import build, qmixer
    build.build()
    qmixer.lib()
    return qmixer


def test_debug_settings_are_checked(M):
    from bit_recurrent_state_decode_b200 import qstate as Q
    f = M.lib().qmixer_debug_set
    assert f(-2, 1) == E and f(0, 0) == E and f(-1, 1 << 24) == 0
    with pytest.raises(Q.QStateError):
        M.debug_set(wait_polls=0)
    M.debug_set()
    assert M.lib().qmixer_scan_timeouts(None, None) == E
