"""The mixer operators at their edges: codes to the bit, values that are not
numbers or leave the range, waits that run out, and calls that have to be refused."""
import pytest
import torch

from bit_recurrent_state_decode_b200 import qmixer as M
from bit_recurrent_state_decode_b200 import qstate as Q

from qmixer_util import half, scan_exact, within

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


# ---------------------------------------------------------------- load
@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("scale_dtype", [Q.F16, Q.F32])
@pytest.mark.parametrize("bits", [2, 4, 6, 8])
def test_load_of_states_that_are_no_numbers(bits, scale_dtype, group):
    """A NaN stays one, for its whole group, and the next step counts it; infinities
    leave the scale that a step's own conversion leaves; other groups are as ever."""
    make = lambda: Q.QState(1, 3, 64, 64, Q.MAMBA2, bits=bits, group=group, scale_dtype=scale_dtype)  # noqa: E731
    obj, clean = make(), make()
    S = normal(gen(bits), 3, 64, 64)
    M.load(clean, S)
    want, (_, scales, _) = clean.dequant(), clean.export()
    want, scales = want.clone(), scales.float().clone()
    S[0, 5, 40], S[1, 7, 33] = float("nan"), -float("inf")
    S[0, 5, 41] = float("inf")                       # beside the NaN, which prevails
    M.load(obj, S)
    got, (_, sc, _) = obj.dequant(), obj.export()
    if group:
        at = [(0, 5, 1), (1, 7, 1)]
        rows = torch.zeros(3, 64, 2, dtype=torch.bool, device=DEV)
        sc, scales = sc.float().view(3, 64, 2), scales.view(3, 64, 2)
    else:
        at = [(0,), (1,)]
        rows = torch.zeros(3, dtype=torch.bool, device=DEV)
        sc, scales = sc.float().view(3), scales.view(3)
    for i in at:
        rows[i] = True
    assert bool(torch.isnan(sc[at[0]]))
    assert float(sc[at[1]]) == (65504.0 if scale_dtype == Q.F16 else float("inf"))
    assert torch.equal(sc[~rows], scales[~rows])
    nan = torch.zeros(3, 64, 64, dtype=torch.bool, device=DEV)
    nan[(0, 5, slice(32, 64)) if group else (0,)] = True
    odd = nan.clone()
    odd[(1, 7, slice(32, 64)) if group else (1,)] = True
    assert bool(torch.isnan(got[nan]).all())
    assert torch.equal(got[~odd], want[~odd])
    # the step behind it sees both tiles (an infinite scale times a code, or a NaN)
    q, k, v, gates, out = obj.alloc_inputs()
    q.fill_(1.0)
    for t in (k, v, gates):
        t.fill_(0.5)
    obj.step(q, k, v, gates, out)
    assert bool(torch.isnan(out[0]).any()) and bool(torch.isfinite(out[2]).all())
    assert obj.status()["nonfinite"] >= 1
    obj.close()
    clean.close()


# ---------------------------------------------------------------- errors behind a launch
CHILD = """
import ctypes, os, sys, torch
from bit_recurrent_state_decode_b200 import qmixer as M, qstate as Q
count = ctypes.c_int.in_dll(ctypes.CDLL(os.environ["LD_PRELOAD"]), "calls")
x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
dt, A = torch.ones(4, 2, device="cuda"), -torch.ones(2, device="cuda")
one, st = torch.ones(1, 2, 64, 64, device="cuda"), torch.ones(4, 2, 64, 64, device="cuda")
c, w = x[:, 0].contiguous(), torch.ones(64, 4, dtype=torch.bfloat16, device="cuda")
c1, cs = torch.ones(1, 3, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(4, 3, 64, dtype=torch.bfloat16, device="cuda")
res = torch.ones_like(c)
calls = [(lambda: M.conv(c, w, state=c1, initial=True), c1), (lambda: M.conv_step(c, w, state=cs), cs),
         (lambda: M.scan(x, dt, A, x, x, state=one, initial=True), one), (lambda: M.scan_step(x, dt, A, x, x, state=st), st),
         (lambda: M.norm(c, w[:, 0].contiguous(), residual=res), res)]
for i, (call, kept) in enumerate(calls):
    before = kept.clone()
    try:
        call()
        sys.exit(f"call {i} was made again")
    except Q.QStateError as e:
        assert e.code == Q.ECUDA, e
    torch.cuda.synchronize()
    assert count.value == i + 1 and torch.equal(kept, before), (i, count.value)
print("once each")
"""


def test_an_error_behind_the_launch_is_raised_and_the_call_not_repeated(tmp_path):
    """C entries that report a CUDA error: the compiled calls raise it after one call.
    (A second one, by way of Python, would move states and residuals on again.)"""
    import os
    import subprocess
    import sys
    names = ("conv", "conv_step", "scan", "scan_step", "norm")
    src, so = tmp_path / "stand_in.c", str(tmp_path / "stand_in.so")
    src.write_text("int calls;\n" + "".join(f"int qmixer_{n}(const void* a, void* s) {{ (void)a; (void)s; calls++; return -3; }}\n"
                                             for n in names))
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", so], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, cwd=root, timeout=300,
                       env={**os.environ, "LD_PRELOAD": so, "PYTHONPATH": root})
    assert r.returncode == 0 and r.stdout.strip() == "once each", r.stdout + r.stderr


# ---------------------------------------------------------------- range of the float32 scan
LARGE = {
    # what is large, and the time step: decays of e^-1.7 leave 2^-40 within 17 tokens
    "x": dict(x=1e30), "x once": dict(x_at=1e30), "B": dict(B=1e31), "C": dict(C=1e33), "state": dict(state=1e33),
    "step": dict(dt=1e20, A=-1.7e-20), "slow": dict(x=1e30, A=-1e-3), "growth": dict(A=2.5, T=30), "just below": dict(x=8191.0, B=8191.0),
}


@pytest.mark.parametrize("T", [16, 70, 2500])
@pytest.mark.parametrize("N,P", [(64, 64), (128, 128)])
@pytest.mark.parametrize("name", sorted(LARGE))
def test_scan_f32_keeps_its_range(name, N, P, T):
    """Inputs, states and steps far beyond a model's under strong decays: every value
    that binary32 holds comes out, long and short, in one piece and cut."""
    kw = LARGE[name]
    T = min(T, kw.get("T", T))
    g = gen(T + N)
    x, B, C = normal(g, T, 1, P) * kw.get("x", 1.0), normal(g, T, 1, N) * kw.get("B", 1.0), normal(g, T, 1, N) * kw.get("C", 1.0)
    if "x_at" in kw:
        x[T // 2] *= kw["x_at"]
    dt = torch.full((T, 1), kw.get("dt", 1.0), device=DEV) * (torch.rand(T, 1, device=DEV, generator=g) + 0.5)
    A = torch.full((1,), kw.get("A", -1.7), device=DEV)
    D = torch.ones(1, device=DEV)
    st = normal(g, 1, 1, N, P) * kw.get("state", 1.0)
    want = scan_exact(x, dt, A, B, C, D, None, False, st, [0, T])
    assert bool((want[4] < 1e38).all())                       # no sum of magnitudes leaves the range
    y = M.scan(x[None], dt[None], A, B[None], C[None], D, softplus=False, state=st, initial=True)
    within("y", y[0], want[0], want[2] + half(F) * (want[0].abs() + want[2]))
    within("state", st, want[1], want[3])


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("what", ["x", "B", "C", "dt"])
def test_scan_f32_large_inputs_reach_no_earlier_token(what, N):
    g = gen(N)
    T, at = 90, 39
    x, B, C = normal(g, T, 2, 64), normal(g, T, 1, N), normal(g, T, 1, N)
    dt, A = torch.rand(T, 2, device=DEV, generator=g), torch.tensor([-1.0, -4.0], device=DEV)
    clean = M.scan(x, dt, A, B, C, softplus=False)
    {"x": x, "B": B, "C": C, "dt": dt}[what][at].view(-1)[1] = 1e9
    assert torch.equal(M.scan(x, dt, A, B, C, softplus=False)[:at], clean[:at])


# ---------------------------------------------------------------- tensors that are refused
def operands():
    g = gen(3)
    x, w = normal(g, 4, 64), normal(g, 64, 4)
    s = dict(x=normal(g, 4, 2, 64), dt=normal(g, 4, 2), A=-torch.rand(2, device=DEV, generator=g), B=normal(g, 4, 2, 64),
             C=normal(g, 4, 2, 64), D=normal(g, 2), dt_bias=normal(g, 2))
    return {
        "conv": (M.conv, dict(x=x, weight=w, bias=w[:, 0].contiguous(), state=normal(g, 1, 3, 64)), dict(initial=True)),
        "conv_step": (M.conv_step, dict(x=x, weight=w, bias=w[:, 0].contiguous(), state=normal(g, 4, 3, 64)), {}),
        "scan": (M.scan, dict(**s, state=normal(g, 1, 2, 64, 64)), dict(initial=True)),
        "scan_step": (M.scan_step, dict(**s, state=normal(g, 4, 2, 64, 64)), {}),
        "norm": (M.norm, dict(x=x, weight=w[:, 0].contiguous(), residual=normal(g, 4, 64)), {}),
        "norm gated": (M.norm, dict(x=x, weight=w[:, 0].contiguous(), gate=normal(g, 4, 64)), {}),
        "load": (lambda S: M.load(obj_of(), S), dict(S=normal(g, 2, 64, 64)), {}),
        "step": (lambda **kw: M.step(obj_of(4), **kw), s, {}),
    }


def obj_of(batch=1):
    return Q.QState(batch, 2, 64, 64, Q.MAMBA2, bits=8, group=32)


@pytest.mark.parametrize("name", ["conv", "conv_step", "scan", "scan_step", "norm", "norm gated", "load", "step"])
def test_tangents_and_negated_views_are_refused(name):
    """An input with a forward-mode tangent would lose it, one with the negative bit
    would be read without its sign: each operand of each operator is refused by name."""
    from torch.autograd import forward_ad
    fn, tensors, kw = operands()[name]
    keep = {n: t.clone() for n, t in tensors.items()}
    for arg, t in tensors.items():
        with forward_ad.dual_level(), pytest.raises(ValueError, match=f"{arg} carries a tangent"):
            fn(**{**tensors, arg: forward_ad.make_dual(t, torch.ones_like(t))}, **kw)
        # the imaginary part of a conjugate view, and the same bit on a dense tensor
        neg = torch._neg_view(t)
        assert neg.is_neg()
        with pytest.raises(ValueError, match=f"{arg} is a view"):
            fn(**{**tensors, arg: neg}, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(tensors[n], keep[n]) for n in tensors), arg
    with forward_ad.dual_level():                             # no tangent: as ever
        fn(**tensors, **kw)


# ---------------------------------------------------------------- waits that run out
@pytest.fixture
def short_waits():
    """Waits of some ten milliseconds; what a test sets is taken back."""
    yield lambda drop: M.debug_set(drop, 1 << 15)
    M.debug_set()


@pytest.mark.parametrize("drop", [0, 1, 2, 3])
@pytest.mark.parametrize("N,P", [(64, 64), (128, 128)])
def test_a_wait_that_runs_out_is_seen(N, P, drop, short_waits):
    """Inputs that never arrive: the call ends, the whole segment is NaN, state and all,
    the block is counted, sequences that ended before are right, and so is the next call."""
    g = gen(drop)
    T = [500, 100]                                           # four chunks and one
    x, B, C = normal(g, 600, 2, P).to(BF), normal(g, 600, 1, N).to(BF), normal(g, 600, 1, N).to(BF)
    dt, A = torch.rand(600, 2, device=DEV, generator=g), torch.tensor([-1.0, -4.0], device=DEV)
    starts = torch.tensor([0, 500, 600], dtype=torch.int32, device=DEV)
    call = lambda: M.scan(x, dt, A, B, C, softplus=False, seq_starts=starts, state=state)  # noqa: E731
    state = torch.zeros(2, 2, N, P, device=DEV)
    want, want_state = call(), state
    before = M.scan_timeouts()
    state = torch.zeros_like(state)
    short_waits(drop)
    y = call()
    M.debug_set()
    after = M.scan_timeouts()
    assert bool(torch.isnan(y[:T[0]]).all()) and bool(torch.isnan(state[0]).all())
    if drop == 0:
        assert bool(torch.isnan(y).all()) and bool(torch.isnan(state).all())
    else:
        assert torch.equal(y[T[0]:], want[T[0]:]) and torch.equal(state[1], want_state[1])
    # two heads of P / 64 blocks each
    assert after - before == (2 if drop == 0 else 1) * 2 * (P // 64)
    state = torch.zeros_like(state)
    assert torch.equal(call(), want) and torch.equal(state, want_state)
    assert M.scan_timeouts() == after


def test_a_wait_that_runs_out_in_a_cut_scan(short_waits):
    """The pass over the segments' states gives up too: what follows is NaN, not a
    number that looks like one."""
    g = gen(4)
    x, B, C = normal(g, 4000, 1, 64).to(BF), normal(g, 4000, 1, 128).to(BF), normal(g, 4000, 1, 128).to(BF)
    dt, A = torch.rand(4000, 1, device=DEV, generator=g) * 0.01, torch.tensor([-1.0], device=DEV)
    assert M.lib().qmixer_scan_workspace(1, 4000, 1, 1, 128, 64, Q.BF16) > 0     # it is cut
    want = M.scan(x, dt, A, B, C, softplus=False)
    before = M.scan_timeouts()
    state = torch.zeros(1, 1, 128, 64, device=DEV)
    short_waits(1)
    y = M.scan(x, dt, A, B, C, softplus=False, state=state)
    M.debug_set()
    assert bool(torch.isnan(y).all()) and bool(torch.isnan(state).all()) and M.scan_timeouts() > before
    assert torch.equal(M.scan(x, dt, A, B, C, softplus=False), want)


# ---------------------------------------------------------------- sizes at the end of their types
@pytest.mark.parametrize("channels", [2 ** 31 - 1, 2 ** 31 - 31])
def test_conv_of_the_most_channels(channels):
    """One token of nearly 2^31 channels: as a prompt and as a step, the ends as those
    of a narrow call."""
    x, w = torch.zeros(1, channels, dtype=BF, device=DEV), torch.zeros(channels, 2, dtype=BF, device=DEV)
    st = torch.zeros(1, 1, channels, dtype=BF, device=DEV)
    g = gen(1)
    for t in (x[0], st[0, 0]):
        t[:99], t[-99:] = normal(g, 99), normal(g, 99)
    w[:99], w[-99:] = normal(g, 99, 2), normal(g, 99, 2)
    ends = lambda t: torch.cat([t[..., :99], t[..., -99:]], -1)  # noqa: E731
    narrow = ends(st)
    want = M.conv(ends(x), torch.cat([w[:99], w[-99:]]), state=narrow, initial=True)
    kept = st.clone()
    assert torch.equal(ends(M.conv(x, w, state=st, initial=True)), want) and torch.equal(ends(st), narrow)
    assert torch.equal(ends(M.conv_step(x, w, state=kept)), want) and torch.equal(ends(kept), narrow)


def overlapping(name):
    """(written operand, the other, a call with the two in one piece of memory): every
    pair of what an operator writes and what it reads."""
    fn, tensors, kw = operands()[name]
    tensors = {n: t.to(F) for n, t in tensors.items()}
    starts = {}
    if name in ("conv", "scan"):
        starts = dict(seq_starts=torch.tensor([0, 4], dtype=torch.int32, device=DEV))
    written = [n for n in ("state", "residual") if n in tensors]
    if "step" != name and name != "load":
        like = tensors["x"]
        tensors = {**tensors, "out": torch.empty_like(like)}
        written.append("out")
    elif name == "step":
        tensors = {**tensors, "out": torch.empty_like(tensors["x"])}
        written.append("out")
    for w in written:
        for other, t in {**tensors, **starts}.items():
            if other == w or (other == "out" and w != "out"):
                continue
            both = torch.zeros(tensors[w].numel() + t.numel(), device=DEV)
            args = {k: v for k, v in tensors.items() if k != "out" or "out" in (w, other)}
            shared = both[:tensors[w].numel()].view(tensors[w].shape)
            # (the other one starts with the last 16 bytes of the written one)
            begin = tensors[w].numel() - 4
            inside = both[begin:begin + t.numel()].view(t.dtype).view(t.shape)
            yield w, other, lambda args=args, w=w, other=other, shared=shared, inside=inside: fn(
                **{**args, **starts, w: shared, other: inside}, **kw)


@pytest.mark.parametrize("name", ["conv", "conv_step", "scan", "scan_step", "norm", "norm gated", "step"])
def test_what_is_written_is_apart_from_what_is_read(name):
    seen = 0
    for w, other, call in overlapping(name):
        with pytest.raises(ValueError, match="overlap"):
            call()
        seen += 1
    assert seen >= 2


def test_a_view_of_one_sequence_is_taken_as_far_as_it_reaches():
    """x of one sequence whose leading stride says nothing about its length."""
    both = torch.zeros(40 * 64 + 3 * 64, device=DEV)
    x = both.as_strided((1, 40, 64), (0, 64, 1))
    w = torch.ones(64, 4, device=DEV)
    M.conv(x, w, state=both[40 * 64:].view(1, 3, 64))
    for out in (None, torch.empty(1, 40, 64, device=DEV)):
        with pytest.raises(ValueError, match="state overlaps x"):
            M.conv(x, w, state=both[20 * 64:23 * 64].view(1, 3, 64), out=out)


# ---------------------------------------------------------------- autograd beside the calls
@pytest.mark.parametrize("name", ["conv", "conv_step", "scan", "scan_step", "norm", "step"])
@pytest.mark.parametrize("given", [False, True])
def test_what_is_written_in_place_is_known_to_autograd(name, given):
    """A product that saved a state or residual for its backward pass is not given the
    values behind the call in their place; inference tensors have no versions."""
    fn, tensors, kw = operands()[name]
    if given:
        tensors["out"] = torch.empty_like(tensors["x"])
    written = [n for n in ("state", "residual", "out") if n in tensors]
    for n in written:
        w = torch.ones_like(tensors[n], requires_grad=True)
        p = (tensors[n] * w).sum()
        fn(**tensors, **kw)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            p.backward()
    for t in (t for n, t in tensors.items() if n not in written):
        assert t._version == 0
    with torch.inference_mode():
        tensors = {n: t.clone() for n, t in tensors.items()}
    fn(**tensors, **kw)


def test_norm_scales_of_the_caller_are_known_to_autograd():
    x, w = normal(gen(1), 4, 64), torch.ones(64, device=DEV)
    scales = torch.ones(4, 1, device=DEV)
    v = scales._version
    M.norm(x, w, dtype=torch.int8, scales=scales)
    assert scales._version == v + 1
