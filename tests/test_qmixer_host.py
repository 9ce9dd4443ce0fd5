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


def call(M, name, **fields):
    import struct
    return getattr(M.lib(), name)(struct.pack(M._FIELDS[name], *fields.values()), None)


@pytest.mark.parametrize("heads,d_v", [(2 ** 30, 128), (2 ** 31 - 1, 128), (2 ** 31 - 1, 64), (65536, 64), (32768, 128)])
def test_more_heads_than_a_grid_are_refused(M, heads, d_v):
    """Also where the number of column parts passes 32 bits."""
    assert M.lib().qmixer_scan_workspace(1, 10, heads, 1, 64, d_v, 1) == U
    row = heads * d_v
    assert call(M, "qmixer_scan", x=4096, x_stride=row, dt=4096, dt_stride=heads, A=4096, B=4096, B_stride=64, C=4096,
                C_stride=64, D=0, dt_bias=0, state=4096, y=4096, y_stride=row, seq_starts=0, sequences=1, tokens=8,
                heads=heads, groups=1, d_k=64, d_v=d_v, dtype=1, dt_dtype=0, flags=4, workspace=4096,
                workspace_bytes=2 ** 40) == U
