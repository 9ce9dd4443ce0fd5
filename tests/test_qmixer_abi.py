"""The C ABI of include/qmixer.h and the argument checks of its binding,
without a GPU: the library exports what the header declares, the argument
structures have the layout the binding packs, invalid calls are refused before
any CUDA call, and the binding refuses what the kernels cannot see."""
import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "bit_recurrent_state_decode_b200")


@pytest.fixture(scope="module")
def M():
    from bit_recurrent_state_decode_b200 import build, qmixer
    build.build()
    qmixer.lib()
    return qmixer


def _header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qmixer.h")).read(), flags=re.S)


def _fields():
    """name -> [(type, field)] of each argument structure in the header."""
    out = {}
    for body, name in re.findall(r"typedef struct \w+ \{(.*?)\} (\w+)_args;", _header(), flags=re.S):
        fields = []
        for line in body.split(";"):
            if not line.strip():
                continue
            first, *more = [t.strip() for t in line.split(",")]
            kind, field = re.match(r"(.*?)(\w+)$", first, flags=re.S).groups()
            fields += [(kind.strip(), f) for f in [field] + more]
        out[name] = fields
    return out


def test_exports_every_declared_symbol(M):
    declared = sorted(set(re.findall(r"\b(qmixer_[a-z_]+)\s*\(", _header())))
    assert sorted(M.EXPORTS) == declared
    for name in declared:
        assert hasattr(M.lib(), name), name


def test_packed_layout_is_the_headers(M):
    code = {"int64_t": "q", "int32_t": "i", "float": "f"}
    fields = _fields()
    assert set(fields) == set(M._FIELDS)
    for name, fs in fields.items():
        assert "".join("P" if "*" in k else code[k] for k, _ in fs) == M._FIELDS[name], name


def test_c_client_agrees_on_sizes_and_gets_answers(M, tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no host compiler")
    sizes = {n: struct.calcsize(f) for n, f in M._FIELDS.items()}
    checks = "\n".join(f"    if (sizeof({n}_args) < {s} || sizeof({n}_args) > {(s + 7) // 8 * 8}) return 10;\n"
                       f"    if ({n}(NULL, NULL) != QSTATE_EINVAL) return 11;" for n, s in sizes.items())
    src = tmp_path / "client.c"
    src.write_text('#include <stdio.h>\n#include "qmixer.h"\nint main(void) {\n' + checks +
                   "\n    if (qmixer_scan_workspace(1, 10, 3, 2, 64, 64, QSTATE_BF16) != QSTATE_EINVAL) return 12;"
                   "\n    if (qmixer_scan_workspace(1, 10, 2, 2, 96, 64, QSTATE_BF16) != QSTATE_EUNSUPPORTED) return 13;"
                   '\n    puts("ok");\n    return 0;\n}\n')
    exe = tmp_path / "client"
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I" + os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe), "-L" + PKG, "-lqmixer", "-Wl,-rpath," + PKG], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip() == "ok"


# ---------------------------------------------------------------- C refusals
GOOD = {
    "qmixer_conv": dict(x=4096, x_stride=64, weight=4096, bias=4096, state=4096, y=8192, y_stride=64, seq_starts=0,
                        sequences=2, tokens=8, channels=64, width=4, dtype=1, flags=3),
    "qmixer_conv_step": dict(x=4096, x_stride=64, weight=4096, bias=0, state=4096, y=8192, y_stride=64, batch=2,
                             channels=64, width=4, dtype=1, flags=2),
    "qmixer_scan": dict(x=4096, x_stride=256, dt=4096, dt_stride=4, A=4096, B=4096, B_stride=128, C=4096, C_stride=128,
                        D=0, dt_bias=0, state=4096, y=8192, y_stride=256, seq_starts=0, sequences=2, tokens=8, heads=4,
                        groups=2, d_k=64, d_v=64, dtype=1, dt_dtype=0, flags=4, workspace=0, workspace_bytes=0),
    "qmixer_scan_step": dict(x=4096, x_stride=256, dt=4096, dt_stride=4, A=4096, B=4096, B_stride=128, C=4096,
                             C_stride=128, D=0, dt_bias=0, state=4096, y=8192, y_stride=256, batch=2, heads=4, groups=2,
                             d_k=64, d_v=64, dtype=1, dt_dtype=0, flags=4),
    "qmixer_step_operands": dict(x=4096, x_stride=256, dt=4096, dt_stride=4, A=4096, B=4096, B_stride=128, C=4096,
                                 C_stride=128, dt_bias=0, q=4096, k=4096, v=4096, gates=4096, batch=2, heads=4,
                                 groups=2, d_k=64, d_v=64, dtype=1, dt_dtype=0, qkv_dtype=0, gate_dtype=0, flags=4),
    "qmixer_step_output": dict(out=4096, x=4096, x_stride=256, D=4096, y=8192, y_stride=256, batch=2, heads=4, d_v=64,
                               dtype=1),
    "qmixer_norm": dict(x=4096, x_stride=64, other=4096, other_stride=64, weight=4096, y=8192, y_stride=64,
                        scales=4096, rows=3, columns=64, group=32, eps=1e-5, dtype=1, before=2, out=1),
    "qmixer_quantize": dict(S=4096, codes=8192, scales=4096, ref=0, rows=2, heads=2, d_k=64, d_v=64, bits=4,
                            head_bits=0, group=32, scale_dtype=2, rotation=0),
}
E, U = -1, -4
BAD = [
    ("qmixer_conv", dict(dtype=2), E), ("qmixer_conv", dict(channels=0), E), ("qmixer_conv", dict(tokens=-1), E),
    ("qmixer_conv", dict(tokens=9), E), ("qmixer_conv", dict(sequences=-1), E), ("qmixer_conv", dict(flags=4), E),
    ("qmixer_conv", dict(x_stride=63), E), ("qmixer_conv", dict(y_stride=0), E), ("qmixer_conv", dict(state=0), E),
    ("qmixer_conv", dict(x=0), E), ("qmixer_conv", dict(x=4097), E), ("qmixer_conv", dict(weight=0), E),
    ("qmixer_conv", dict(width=5), U), ("qmixer_conv", dict(width=1), U), ("qmixer_conv", dict(tokens=2 ** 31), E),
    ("qmixer_conv_step", dict(state=0), E), ("qmixer_conv_step", dict(flags=1), E), ("qmixer_conv_step", dict(width=9), U),
    ("qmixer_scan", dict(groups=3), E), ("qmixer_scan", dict(groups=0), E), ("qmixer_scan", dict(heads=0), E),
    ("qmixer_scan", dict(d_k=32), U), ("qmixer_scan", dict(d_v=256, x_stride=1024, y_stride=1024), U), ("qmixer_scan", dict(x_stride=260), E),
    ("qmixer_scan", dict(B=4104), E), ("qmixer_scan", dict(flags=2), E), ("qmixer_scan", dict(flags=5, state=0), E),
    ("qmixer_scan", dict(dt_dtype=2), E), ("qmixer_scan", dict(tokens=7), E), ("qmixer_scan", dict(A=0), E),
    ("qmixer_scan", dict(dt_stride=3), E), ("qmixer_scan", dict(state=4100), E), ("qmixer_scan", dict(C_stride=120), E),
    # one long prompt of few heads is cut into segments, which need room
    ("qmixer_scan", dict(sequences=1, tokens=100000), E),
    ("qmixer_scan", dict(sequences=1, tokens=100000, workspace=4096, workspace_bytes=1024), E),
    ("qmixer_scan_step", dict(state=0), E), ("qmixer_scan_step", dict(y=0), E), ("qmixer_scan_step", dict(d_k=16), U),
    ("qmixer_scan_step", dict(batch=-1), E), ("qmixer_scan_step", dict(flags=1), E),
    ("qmixer_step_operands", dict(q=0), E), ("qmixer_step_operands", dict(qkv_dtype=2), E),
    ("qmixer_step_operands", dict(gates=4098), E),
    ("qmixer_step_output", dict(x=0), E), ("qmixer_step_output", dict(y_stride=255), E),
    ("qmixer_norm", dict(group=24), E), ("qmixer_norm", dict(columns=96, x_stride=96, y_stride=96, other_stride=96, group=48), U),
    ("qmixer_norm", dict(columns=0), E), ("qmixer_norm", dict(eps=-1.0), E), ("qmixer_norm", dict(eps=float("nan")), E),
    ("qmixer_norm", dict(before=3), E), ("qmixer_norm", dict(out=3), E), ("qmixer_norm", dict(out=0), E),
    ("qmixer_norm", dict(other=0), E), ("qmixer_norm", dict(scales=0), E), ("qmixer_norm", dict(rows=-1), E),
    ("qmixer_norm", dict(columns=40000, x_stride=40000, y_stride=40000, other_stride=40000, group=0), U),
    ("qmixer_quantize", dict(bits=5), E), ("qmixer_quantize", dict(group=12), E), ("qmixer_quantize", dict(d_k=96), U),
    ("qmixer_quantize", dict(scale_dtype=1), E), ("qmixer_quantize", dict(rotation=2), E),
    ("qmixer_quantize", dict(scales=0), E), ("qmixer_quantize", dict(codes=8200), E), ("qmixer_quantize", dict(rows=2 ** 31), E),
]


def _call(M, name, fields):
    return getattr(M.lib(), name)(struct.pack(M._FIELDS[name], *fields.values()), None)


@pytest.mark.parametrize("name", sorted(GOOD))
def test_the_base_of_the_refusals_names_every_field(M, name):
    assert list(GOOD[name]) == [f for _, f in _fields()[name]]


@pytest.mark.parametrize("name,change,code", BAD)
def test_invalid_calls_are_refused_before_cuda(M, name, change, code):
    assert set(change) <= set(GOOD[name])
    assert _call(M, name, {**GOOD[name], **change}) == code


@pytest.mark.parametrize("name,change", [
    ("qmixer_conv", dict(sequences=0, tokens=0)), ("qmixer_conv_step", dict(batch=0)),
    ("qmixer_scan", dict(sequences=0, tokens=0)), ("qmixer_scan_step", dict(batch=0)),
    ("qmixer_step_operands", dict(batch=0)), ("qmixer_step_output", dict(batch=0)), ("qmixer_norm", dict(rows=0)),
    ("qmixer_quantize", dict(rows=0))])
def test_empty_calls_do_nothing(M, name, change):
    assert _call(M, name, {**GOOD[name], **change}) == 0


def test_bad_head_bits(M):
    hb = (ctypes.c_uint8 * 2)(4, 5)
    assert _call(M, "qmixer_quantize", {**GOOD["qmixer_quantize"], "head_bits": ctypes.addressof(hb)}) == E


def test_workspace(M):
    w = M.lib().qmixer_scan_workspace
    assert w(0, 0, 4, 1, 64, 64, 1) == 0
    assert w(1, -1, 4, 1, 64, 64, 1) == E
    assert w(1, 8, 4, 1, 64, 64, 2) == E
    assert w(1, 8, 4, 1, 64, 80, 1) == U
    assert w(1, 100000, 4, 1, 64, 64, 1) > 0


# ---------------------------------------------------------------- binding refusals
def test_host_tensors_are_refused(M):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        M.conv(x, torch.zeros(64, 4))
    with pytest.raises(ValueError, match="CUDA"):
        M.conv_step(x, torch.zeros(64, 4), state=torch.zeros(4, 3, 64))
    with pytest.raises(ValueError, match="CUDA"):
        M.norm(x, torch.zeros(64))
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        M.scan(x, torch.zeros(4, 2), torch.zeros(2), x, x)
    with pytest.raises(ValueError, match="CUDA"):
        M.scan_step(x, torch.zeros(4, 2), torch.zeros(2), x, x, state=torch.zeros(4, 2, 64, 64))


def test_row_strides(M):
    t = torch.zeros(6, 4, 10)
    assert M._rows("f", "t", t, 1) == 10
    assert M._rows("f", "t", t, 2) == 40
    assert M._rows("f", "t", t[0, :, :4], 1) == 10
    assert M._rows("f", "t", torch.zeros(3, 5, 8)[:, :, :6], 1) == 8      # sequences one behind the other
    assert M._rows("f", "t", t[:, :1, :6], 1) == 40                        # one token of each sequence
    assert M._rows("f", "t", torch.zeros(0, 7), 1) == 7
    for bad in (t[:, :3], t.transpose(0, 1), t[..., ::2], torch.zeros(1, 10).expand(4, 10), t[::2, :3]):
        with pytest.raises(ValueError):
            M._rows("f", "t", bad, 1)
    with pytest.raises(ValueError):
        M._rows("f", "t", t[..., :6], 2)


def test_overlaps(M):
    b = torch.zeros(8, 32)
    M._apart("f", "out", b[:4], "x", b[4:])
    M._apart("f", "out", b[:, :16], "x", b[:, 16:])        # columns of one buffer's rows
    M._apart("f", "out", b, "x", torch.zeros(8, 32))
    M._apart("f", "out", b[:0], "x", b)
    c = b.view(2, 4, 32)
    M._apart("f", "out", c[..., :16], "x", c[..., 16:])
    M._apart("f", "out", c[..., :16].unflatten(-1, (4, 4)), "x", c[..., 16:24])
    with pytest.raises(ValueError):
        M._apart("f", "out", c[..., :16], "x", c[..., 8:24])
    for other in (b, b[2:6], b[:, 15:], b.view(16, 16)):
        with pytest.raises(ValueError):
            M._apart("f", "out", b[:, :16] if other.shape[-1] == 17 else b, "x", other)


def test_gradients_are_refused(M):
    t = torch.zeros(4, requires_grad=True)

    class Fake(torch.Tensor):
        def get_device(self):
            return 0
    f = t.as_subclass(Fake)
    with pytest.raises(ValueError, match="gradient"):
        M._tensor("f", "t", f, 0)
    with torch.no_grad():
        M._tensor("f", "t", f, 0)
