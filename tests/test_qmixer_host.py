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


# ---------------------------------------------------------------- the build
def child(code):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)


def test_the_libraries_build_without_pytorch(M):
    """A C user has nvcc alone: nothing of the build may need PyTorch but the module
    that only Python loads."""
    r = child("import sys; sys.modules['torch'] = None\n"
              "from bit_recurrent_state_decode_b200 import build\n"
              "print(build.build() == build.LIB, build.up_to_date())\n"
              "build._build_usual()")
    assert r.returncode == 0 and r.stdout.split() == ["True", "True"], r.stdout + r.stderr
    assert "left out" in r.stderr


def test_a_module_for_other_versions_is_built_again_and_not_loaded(M, monkeypatch):
    from bit_recurrent_state_decode_b200 import build
    assert build._usual_up_to_date() and build.usual_built_for(build.usual_versions())
    monkeypatch.setattr(build, "usual_versions", lambda: "cpython-399 torch 99.0")
    assert not build._usual_up_to_date() and not build.up_to_date()
    with pytest.raises(RuntimeError, match="other versions"):
        M._Load().norm


# ---------------------------------------------------------------- the plan of a cut prompt
@pytest.mark.parametrize("sequences,tokens,H,N,P,dtype,ragged,segments", [
    (1, 16001, 16, 128, 128, 1, False, 9),           # nine of 1792 tokens
    (7, 3001, 16, 64, 64, 0, True, 3001 // 64 + 7),  # of 64 tokens, and room for each sequence's last
    (8, 16384, 32, 128, 64, 1, False, 0),            # uncut
    (8, 8192, 32, 128, 64, 0, False, 0),
])
@pytest.mark.skipif(torch.cuda.is_available(), reason="the last call would launch")
def test_plan_of_the_documented_sizes(M, sequences, tokens, H, N, P, dtype, ragged, segments):
    """The least workspace that a call takes is that of the segments which the comments
    and tables name (148 SMs)."""
    need = segments * H * N * P * 4 + (segments * H * 4 + 15) // 16 * 16
    starts = 4096 if ragged else 0

    def rc(size):
        return call(M, "qmixer_scan", x=4096, x_stride=H * P, dt=4096, dt_stride=H, A=4096, B=4096, B_stride=N, C=4096,
                    C_stride=N, D=0, dt_bias=0, state=0, y=4096, y_stride=H * P, seq_starts=starts, sequences=sequences,
                    tokens=tokens, heads=H, groups=1, d_k=N, d_v=P, dtype=dtype, dt_dtype=0, flags=4, workspace=4096,
                    workspace_bytes=size)
    assert M.lib().qmixer_scan_workspace(sequences, tokens, H, 1, N, P, dtype) >= need
    assert rc(need) == -3                            # as far as the launch, for which there is no GPU
    if need:
        assert rc(need - 1) == E
