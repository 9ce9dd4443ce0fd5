"""The mixer operators at their edges: codes to the bit, values that are not
numbers or leave the range, waits that run out, and calls that have to be refused."""
import pytest
import torch

from bit_recurrent_state_decode_b200 import qmixer as M
from bit_recurrent_state_decode_b200 import qstate as Q

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_recurrent_state_decode_b200 import build
    build.build()
    assert torch.cuda.is_available()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("before", ["none", "residual"])
@pytest.mark.parametrize("rows,columns,group", [(700, 2048, 0), (1300, 2048, 128), (3, 4096, 32), (1, 1024, 8), (300, 1001, 0)])
def test_norm_codes_to_the_bit(rows, columns, group, before, dtype):
    """The scale is the rounded quotient of the maximum, the code the rounding of the
    quotient by it: from the kernel's own binary32 values, which the same rows
    give as float32 output (bfloat16 rows hold the same numbers)."""
    g = gen(columns + group)
    x, o = normal(g, rows, columns).to(dtype), normal(g, rows, columns).to(dtype)
    x[0] *= 1e-20                                    # eps outweighs it: scales near 1e-20
    w = (torch.rand(columns, device=DEV, generator=g) + 0.5).to(dtype)
    given = lambda t: {} if before == "none" else {before: t.clone()}  # noqa: E731
    y = M.norm(x.float(), w.float(), **given(o.float()))
    parts = y.view(rows, -1, group or columns)
    for to, most in ((torch.int8, 127.0), (torch.float8_e4m3fn, 448.0)):
        codes, scales = M.norm(x, w, dtype=to, group=group, **given(o))
        # (a binary64 quotient of two binary32 numbers rounds to their binary32 one)
        want = (parts.abs().amax(-1).double() / most).float()
        assert torch.equal(scales, want.view_as(scales))
        z = (parts.double() / want.double()[..., None]).float().clamp(-most, most)
        want = z.round().to(torch.int8) if to is torch.int8 else z.to(torch.float8_e4m3fn)
        assert torch.equal(codes.float(), want.float().view_as(codes))


@pytest.mark.parametrize("to,most", [(torch.int8, 127), (torch.float8_e4m3fn, 448.0)])
def test_norm_codes_of_the_smallest_rows(to, most):
    """Scales below the normal numbers: clamped codes, zeros for zeros, no other value."""
    x = torch.zeros(4, 64, device=DEV)
    x[0, ::2], x[1], x[2, 3] = 1e-38, 1e-40, -3e-42
    y = M.norm(x, torch.ones(64, device=DEV), eps=1.0)
    codes, scales = M.norm(x, torch.ones(64, device=DEV), eps=1.0, dtype=to)
    want = (y.abs().amax(-1, keepdim=True).double() / most).float()
    assert torch.equal(scales, want)
    z = torch.where(want > 0, (y.double() / want.double()).float().clamp(-most, most), 0.0)
    want = z.round().to(torch.int8) if to is torch.int8 else z.to(torch.float8_e4m3fn)
    assert torch.equal(codes.float(), want.float())
