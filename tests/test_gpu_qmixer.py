"""The mixer operators on the GPU against their definitions in 64 bits
(qmixer_util): sizes from one token up, odd and strided rows, empty and ragged
sequences, non-finite inputs, streams and graphs, and a layer's run of them
together, on float32 and on low-bit states."""
import pytest
import torch

from bit_recurrent_state_decode_b200 import qmixer as M
from bit_recurrent_state_decode_b200 import qstate as Q

from qmixer_util import U, conv_exact, half, norm_exact, rel2, scan_exact, within

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


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- convolution
CONV = [
    # starts, channels, width
    ([0, 1], 8, 4), ([0, 2], 8, 2), ([0, 5, 5, 6, 6, 9], 24, 4), ([0, 15, 17, 33], 64, 4), ([0, 16, 32, 48], 40, 3),
    ([0, 100], 2304, 4), ([0, 0, 0], 16, 4), ([0, 31, 32, 33, 34, 35, 200], 13, 3), ([3, 20, 21, 64], 8, 4),
    ([0, 257], 1, 2),
]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("starts,channels,width", CONV)
def test_conv(starts, channels, width, initial, dtype):
    g = gen(len(starts) + channels)
    n, T = len(starts) - 1, starts[-1] + 7                       # seven rows behind the last sequence
    x, w = normal(g, T, channels).to(dtype), normal(g, channels, width).to(dtype)
    b, st = normal(g, channels).to(dtype), normal(g, n, width - 1, channels).to(dtype)
    zero = torch.zeros_like(st)
    for act in (True, False):
        y, want, e = conv_exact(x, w, b, st if initial else zero, starts, act)
        state, out = st.clone(), torch.full_like(x, 7.0)
        got = M.conv(x, w, b, state=state, initial=initial, seq_starts=ints(starts), activation=act, out=out)
        assert got is out
        s = slice(starts[0], starts[-1])
        within("y", got[s], y[s], e[s] + half(dtype) * (y[s].abs() + e[s]))
        assert torch.equal(state.double(), want)                   # rows are moved, not computed
        assert bool((out[:starts[0]] == 7).all()) and bool((out[starts[-1]:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F])
def test_conv_batch_strided_and_without_state(dtype):
    g = gen(5)
    wide = normal(g, 3, 50, 96).to(dtype)
    for cols in (slice(8, 72), slice(3, 30)):                     # on and off a 16-byte boundary
        x = wide[..., cols]
        C = x.shape[-1]
        w = normal(g, C, 4).to(dtype)
        y, _, e = conv_exact(x.reshape(150, C), w, None, torch.zeros(3, 3, C, device=DEV), [0, 50, 100, 150], True)
        out = torch.zeros(3, 50, 96, dtype=dtype, device=DEV)
        M.conv(x, w, out=out[..., cols])
        within("y", out[..., cols].reshape(150, C), y, e + half(dtype) * (y.abs() + e))
        out[..., cols] = 0
        assert not bool(out.any())


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("batch,channels,width", [(1, 8, 4), (3, 13, 2), (64, 2304, 4), (5, 100, 3)])
def test_conv_step_moves_on_by_one(batch, channels, width, dtype):
    g = gen(batch + channels)
    x, w = normal(g, batch, channels).to(dtype), normal(g, channels, width).to(dtype)
    b, st = normal(g, channels).to(dtype), normal(g, batch, width - 1, channels).to(dtype)
    y, want, e = conv_exact(x, w, b, st, list(range(batch + 1)), True)
    got = M.conv_step(x, w, b, state=st)
    within("y", got, y, e + half(dtype) * (y.abs() + e))
    assert torch.equal(st.double(), want)


def test_conv_in_pieces_is_conv_in_one():
    """A prompt in three pieces, then single tokens: bit for bit the one call."""
    g = gen(9)
    x, w, b = normal(g, 1, 70, 128).to(BF), normal(g, 128, 4).to(BF), normal(g, 128).to(BF)
    whole = torch.zeros(1, 3, 128, dtype=BF, device=DEV)
    y = M.conv(x, w, b, state=whole)
    st = torch.full_like(whole, float("nan"))                      # not read by the first piece
    parts = [M.conv(x[:, :33], w, b, state=st), M.conv(x[:, 33:35], w, b, state=st, initial=True),
             M.conv(x[:, 35:68], w, b, state=st, initial=True)]
    parts += [M.conv_step(x[:, t], w, b, state=st)[:, None] for t in (68, 69)]
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(st, whole)


def test_conv_causal_with_nonfinite_rows():
    g = gen(3)
    x, w = normal(g, 40, 16), normal(g, 16, 4)
    clean = M.conv(x, w)
    x[20, 3], x[21, 5] = float("nan"), float("inf")
    got = M.conv(x, w)
    keep = torch.ones_like(x, dtype=torch.bool)
    keep[20:24, 3] = keep[21:25, 5] = False
    assert torch.equal(got[keep], clean[keep])
    assert bool(torch.isnan(got[20:24, 3]).all())


# ---------------------------------------------------------------- selective scan
def selective(g, T, H, G, N, P, dtype, dt_dtype=None, view=False):
    pre = normal(g, T, H * P + 2 * G * N)
    mixed = (pre * torch.sigmoid(pre)).to(dtype)
    x, B, C = mixed.split([H * P, G * N, G * N], -1)
    x, B, C = x.unflatten(-1, (H, P)), B.unflatten(-1, (G, N)), C.unflatten(-1, (G, N))
    if not view:
        x, B, C = x.contiguous(), B.contiguous(), C.contiguous()
    dt = normal(g, T, H).to(dt_dtype or dtype)
    A = -torch.rand(H, device=DEV, generator=g) * 15 - 1
    step = torch.exp(torch.rand(H, device=DEV, generator=g) * 4.6 - 6.9)
    return x, dt, A, B, C, torch.rand(H, device=DEV, generator=g), torch.log(torch.expm1(step))


def check_scan(y, state, want, dtype, rows=slice(None)):
    yw, S, ey, eS, most = want
    yw, ey, most = yw[rows], ey[rows], most[rows]
    # bfloat16: the output's rounding, and one of each factor of two products
    # (M, S), relative to their terms
    factor = 2 * half(BF) * most if dtype == BF else 0.0
    within("y", y[rows], yw, ey + factor + half(dtype) * (yw.abs() + ey))
    if dtype == BF and yw.numel() > 4096:
        # three independent roundings of at most half a step: 2^-8 / sqrt(3) each
        assert rel2(y[rows], yw) <= 2.0 ** -8
    if state is not None:
        within("state", state, S, eS)
        assert rel2(state, S) <= 2e-6


SCAN = [
    # starts, heads, groups, d_k, d_v
    ([0, 1], 1, 1, 64, 64), ([0, 1, 2, 3], 2, 1, 128, 64), ([0, 127], 2, 2, 64, 128), ([0, 128], 2, 1, 128, 128),
    ([0, 129], 3, 1, 128, 64), ([0, 37, 37, 300, 301], 4, 2, 128, 64), ([0, 0, 0], 2, 1, 64, 64),
    ([5, 260, 400], 2, 1, 64, 64), ([0, 256, 512, 768], 5, 5, 128, 128), ([0, 16, 31, 47, 64], 2, 1, 64, 64),
    ([0, 3001], 1, 1, 128, 64),          # one long chain: cut into segments
    ([0, 1999, 2000, 2000, 3300], 2, 1, 64, 128),
]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("starts,H,G,N,P", SCAN)
def test_scan(starts, H, G, N, P, initial, dtype):
    g = gen(starts[-1] + H + N)
    n, T = len(starts) - 1, starts[-1] + 9
    x, dt, A, B, C, D, bias = selective(g, T, H, G, N, P, dtype, view=True)
    st = normal(g, n, H, N, P) * 0.3
    want = scan_exact(x, dt, A, B, C, D, bias, True, st if initial else torch.zeros_like(st), starts)
    state, out = st.clone(), torch.full((T, H, P), 7.0, dtype=dtype, device=DEV)
    # what lies behind the last sequence, or in front of the first, is never read
    for t in (x, dt, B, C):
        t[starts[-1]:] = float("nan")
        t[:starts[0]] = float("nan")
    M.scan(x, dt, A, B, C, D, dt_bias=bias, state=state, initial=initial, seq_starts=ints(starts), out=out)
    check_scan(out, state, want, dtype, slice(starts[0], starts[-1]))
    assert bool((out[:starts[0]] == 7).all()) and bool((out[starts[-1]:] == 7).all())


@pytest.mark.parametrize("dtype,dt_dtype", [(BF, F), (F, BF), (BF, BF)])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_batch_types_and_plain_steps(dtype, dt_dtype, softplus):
    g = gen(4)
    n, L, H, G, N, P = 3, 140, 4, 2, 64, 64
    x, dt, A, B, C, D, bias = selective(g, n * L, H, G, N, P, dtype, dt_dtype)
    if not softplus:
        dt, bias = (dt.float().abs() * 0.05).to(dt_dtype), None
    starts = [0, L, 2 * L, 3 * L]
    want = scan_exact(x, dt, A, B, C, None, bias, softplus, torch.zeros(n, H, N, P, device=DEV), starts)
    state = torch.full((n, H, N, P), float("nan"), device=DEV)
    by = [t.view(n, L, *t.shape[1:]) for t in (x, dt, B, C)]
    y = M.scan(by[0], by[1], A, by[2], by[3], dt_bias=bias, softplus=softplus, state=state)
    check_scan(y.view(n * L, H, P), state, want, dtype)
    # without a state to keep: the same outputs
    assert torch.equal(M.scan(by[0], by[1], A, by[2], by[3], dt_bias=bias, softplus=softplus), y)


@pytest.mark.parametrize("dtype", [BF, F])
def test_scan_decays_from_none_to_all(dtype):
    """Decays of exactly one, decays that underflow to zero, and time steps of zero."""
    g = gen(8)
    T, H, N, P = 300, 4, 64, 64
    x, dt, _, B, C, D, _ = selective(g, T, H, 1, N, P, dtype, F)
    A = torch.tensor([0.0, -1e4, -1.0, -16.0], device=DEV)
    dt = torch.rand(T, H, device=DEV, generator=g)
    dt[::7] = 0.0
    dt[100:103] = 300.0
    dt *= 0.02
    want = scan_exact(x, dt, A, B, C, D, None, False, torch.ones(1, H, N, P, device=DEV), [0, T])
    state = torch.ones(1, H, N, P, device=DEV)
    y = M.scan(x[None], dt[None], A, B[None], C[None], D, softplus=False, state=state, initial=True)
    check_scan(y[0], state, want, dtype)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("what", ["x", "B", "C", "dt"])
def test_scan_nonfinite_inputs_reach_no_earlier_token(what, dtype):
    g = gen(6)
    T, H, N, P, at = 300, 2, 64, 128, 200
    x, dt, A, B, C, D, bias = selective(g, T, H, 1, N, P, dtype)
    clean = M.scan(x, dt, A, B, C, D, dt_bias=bias)
    {"x": x, "B": B, "C": C, "dt": dt}[what][at].view(-1)[1] = float("inf") if what == "x" else float("nan")
    y = M.scan(x, dt, A, B, C, D, dt_bias=bias)
    assert torch.equal(y[:at], clean[:at])
    if what == "x":             # its own column, from its token on, and no other
        assert not bool(torch.isfinite(y[at:, 0, 1]).any())
        y[at:, 0, 1] = clean[at:, 0, 1] = 0
        assert torch.equal(y, clean)
    else:
        assert not bool(torch.isfinite(y[at]).all())


@pytest.mark.parametrize("dtype", [BF, F])
def test_scan_starts_out_of_range_touch_nothing_else(dtype):
    """Bounds are clamped and descending starts write inside the buffers only."""
    g = gen(2)
    T, H, N, P = 200, 2, 64, 64
    x, dt, A, B, C, D, bias = selective(g, T, H, 1, N, P, dtype)
    for starts in ([-5, 90, 10 ** 6], [0, 200, 0, 200, 0, 200], [150, 20, 7]):
        n = len(starts) - 1
        pad = torch.full((n + 2, H, N, P), 5.0, device=DEV)
        buf = torch.full((T + 64, H, P), 5.0, dtype=dtype, device=DEV)
        M.scan(x, dt, A, B, C, D, dt_bias=bias, state=pad[1:-1], seq_starts=ints(starts), out=buf[32:-32])
        M.conv(x.view(T, -1), torch.ones(H * P, 4, dtype=dtype, device=DEV), seq_starts=ints(starts),
               state=torch.zeros(n, 3, H * P, dtype=dtype, device=DEV), out=buf[32:-32].view(T, -1))
        torch.cuda.synchronize()
        assert bool((pad[0] == 5).all()) and bool((pad[-1] == 5).all())
        assert bool((buf[:32] == 5).all()) and bool((buf[-32:] == 5).all())
    y = M.scan(x, dt, A, B, C, D, dt_bias=bias, seq_starts=ints([-5, 90, 10 ** 6]))
    assert torch.equal(y, M.scan(x, dt, A, B, C, D, dt_bias=bias, seq_starts=ints([0, 90, T])))


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,H,G,N,P", [(1, 1, 1, 64, 64), (3, 4, 2, 128, 64), (2, 5, 1, 64, 128), (7, 2, 2, 128, 128)])
def test_scan_step(n, H, G, N, P, dtype):
    g = gen(n + H)
    x, dt, A, B, C, D, bias = selective(g, n, H, G, N, P, dtype, view=True)
    st = normal(g, n, H, N, P)
    yw, S, ey, eS, most = scan_exact(x, dt, A, B, C, D, bias, True, st, list(range(n + 1)))
    y = M.scan_step(x, dt, A, B, C, D, dt_bias=bias, state=st)
    within("y", y, yw, ey + half(dtype) * (yw.abs() + ey))          # no factor is rounded here
    within("state", st, S, eS)
    assert rel2(st, S) <= 2e-7


def test_scan_step_offsets_past_32_bits():
    """States past 2^31 elements: the last row of a large batch."""
    n, H, N, P = 2 ** 31 // (64 * 128 * 128) + 3, 64, 128, 128
    g = gen(1)
    x, dt, A, B, C, D, bias = selective(g, n, H, 1, N, P, BF)
    st = torch.empty(n, H, N, P, device=DEV)
    st[-1].normal_(generator=g)
    last = st[-1:].clone()
    y = M.scan_step(x, dt, A, B, C, D, dt_bias=bias, state=st)
    assert torch.equal(y[-1:], M.scan_step(x[-1:], dt[-1:], A, B[-1:], C[-1:], D, dt_bias=bias, state=last))
    assert torch.equal(st[-1:], last)


# ---------------------------------------------------------------- the low-bit state
def codes_of(S, bits, group, scale_dtype):
    """(values, scales) of the dynamic rule, decided in 64 bits."""
    most = 2.0 ** (bits - 1) - 1
    parts = S.double().reshape(len(S), -1, group) if group else S.double().reshape(len(S), 1, -1)
    scale = (parts.abs().amax(-1) / most).float()
    if scale_dtype == Q.F16:
        scale = scale.half().float().clamp(max=65504.0)
    inv = torch.where(scale > 0, 1 / scale, torch.zeros_like(scale))
    c = torch.clamp(torch.round(parts * inv.double()[..., None]), -most, most)
    return (c.float() * scale[..., None]).view_as(S), scale


@pytest.mark.parametrize("bits", [2, 4, 6, 8])
@pytest.mark.parametrize("group", [0, 8, 32, 64])
@pytest.mark.parametrize("scale_dtype", [Q.F16, Q.F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_load_is_the_dynamic_rule_bit_for_bit(bits, group, scale_dtype, dk, dv):
    g = gen(bits + group)
    obj = Q.QState(2, 3, dk, dv, Q.MAMBA2, bits=bits, group=group, scale_dtype=scale_dtype)
    S = normal(g, 6, dk, dv) * 0.3
    S[1] = 0                                                       # a tile without a scale
    S[2, 0] = torch.arange(dv, device=DEV) * 0.5                   # ties
    S[3] = 1e-42                                                   # below the normal numbers
    M.load(obj, S)
    values, scale = codes_of(S, bits, group, scale_dtype)
    _, scales, _ = obj.export()
    assert torch.equal(scales.float().view_as(scale), scale)
    assert torch.equal(obj.dequant(), values)
    obj.close()


def test_load_mixed_widths_yoked_rotated_and_wide():
    g = gen(12)
    hb = [2, 4, 6, 8, 4]
    obj = Q.QState(3, 5, 128, 64, Q.GDN, group=32, scale_mode=Q.YOKED, head_bits=hb, scale_dtype=Q.F32)
    S = normal(g, 3, 5, 128, 64)
    M.load(obj, S)
    got = obj.dequant().view(3, 5, 128, 64)
    for h, b in enumerate(hb):
        assert torch.equal(got[:, h], codes_of(S[:, h].contiguous(), b, 32, Q.F32)[0]), h
    assert torch.equal(obj.export()[2].view_as(S), S)              # the reference is the state itself
    obj.close()
    # rotated: the Hadamard butterfly along d_v, then the rule
    obj = Q.QState(1, 2, 64, 128, Q.GDN, bits=4, group=32, rotation=1)
    S = normal(g, 2, 64, 128)
    R, s = S.clone(), 1
    while s < 128:
        v = R.view(2, 64, 128 // (2 * s), 2, s)
        R = torch.stack([v[..., 0, :] + v[..., 1, :], v[..., 0, :] - v[..., 1, :]], -2).view(2, 64, 128)
        s *= 2
    M.load(obj, S)
    assert torch.equal(obj.dequant(), codes_of(R, 4, 32, Q.F16)[0])
    obj.close()
    # 32 bits: a copy
    obj = Q.QState(1, 2, 64, 64, Q.RETNET, bits=32)
    S = normal(g, 2, 64, 64)
    M.load(obj, S)
    assert torch.equal(obj.dequant(), S)
    obj.close()


def test_load_groups_of_a_whole_row():
    obj = Q.QState(1, 1, 64, 128, Q.MAMBA2, bits=4, group=128)
    S = normal(gen(1), 1, 64, 128)
    M.load(obj, S)
    assert torch.equal(obj.dequant(), codes_of(S, 4, 128, Q.F16)[0])
    obj.close()


def test_load_empties_a_bypass_and_refuses_rowcol():
    S = normal(gen(1), 2, 64, 64)
    obj = Q.QState(1, 2, 64, 64, Q.MAMBA2, bits=4, group=32)
    obj.set_lrb(1, 3, 0.5)
    q, k, v, gates, out = obj.alloc_inputs()
    for t in (q, k, v):
        t.normal_()
    gates.fill_(0.9)
    obj.step(q, k, v, gates, out)
    M.load(obj, S)
    assert torch.equal(obj.dequant(), codes_of(S, 4, 32, Q.F16)[0]) and not bool(obj.lrb_export()["n"].any())
    obj.close()
    obj = Q.QState(1, 2, 64, 64, Q.MAMBA2, bits=4, group=0)
    obj.set_rowcol()
    with pytest.raises(ValueError, match="row x column"):
        M.load(obj, S)
    obj.close()


@pytest.mark.parametrize("qkv,gate", [(Q.F32, Q.F32), (Q.BF16, Q.F32), (Q.BF16, Q.BF16)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_step_on_a_low_bit_state(dtype, qkv, gate):
    """step = the operands from their definition, qstate_step, and D x."""
    g = gen(21)
    n, H, G, N, P = 3, 4, 2, 128, 64
    make = lambda: Q.QState(n, H, N, P, Q.MAMBA2, bits=8, group=0, qkv_dtype=qkv, gate_dtype=gate)  # noqa: E731
    a, b = make(), make()
    S = normal(g, n * H, N, P)
    M.load(a, S)
    M.load(b, S)
    x, dt, A, B, C, D, bias = selective(g, n, H, G, N, P, dtype, view=True)
    y = M.step(a, x, dt, A, B, C, D, dt_bias=bias)
    z = dt.double() + bias.double()
    d = torch.nn.functional.softplus(z, threshold=700.0)
    q, k, v, gates, out = b.alloc_inputs()
    q.copy_(C.repeat_interleave(H // G, 1).reshape(n * H, N))
    k.copy_(B.repeat_interleave(H // G, 1).reshape(n * H, N))
    # dt is off by a few units, so v and the gate may differ by one rounding
    v.copy_((d[..., None] * x.double()).reshape(n * H, P))
    gates.copy_(torch.exp(d * A.double()).reshape(n * H, 1))
    b.step(q, k, v, gates, out)
    ref = out.view(n, H, P).double() + D.double()[:, None] * x.double()
    # one step of 8-bit codes is what a rounding of v or the gate may move
    slack = (half(BF) if Q.BF16 in (qkv, gate) else 64 * U) * 8
    scale = out.abs().amax().double() + ref.abs()
    within("y", y, ref, slack * scale + half(dtype) * ref.abs())
    da, db = a.dequant(), b.dequant()
    step = S.abs().amax() / 127
    assert float((da - db).abs().max()) <= 1.01 * float(step) + slack * float(db.abs().max())
    a.close()
    b.close()


# ---------------------------------------------------------------- norm
NORM = [(1, 1), (3, 7), (2, 8), (5, 256), (1, 264), (61, 2048), (1300, 2048), (1300, 1000), (7, 1025), (1200, 513),
        (2, 4096), (3, 8192), (1, 9000), (2, 16384), (1, 32768), (2, 32761)]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("before", ["none", "residual", "gate"])
@pytest.mark.parametrize("rows,columns", NORM)
def test_norm(rows, columns, before, dtype):
    g = gen(rows + columns)
    x, o = normal(g, rows, columns).to(dtype), normal(g, rows, columns).to(dtype)
    w = (torch.rand(columns, device=DEV, generator=g) + 0.5).to(dtype)
    res, gate = (o if before == "residual" else None), (o if before == "gate" else None)
    y, h, rel = norm_exact(x, w, res, gate, 1e-5)
    kw = {} if before == "none" else {before: o.clone()}
    got = M.norm(x, w, **kw)
    within("y", got, y, (rel + half(dtype)) * 1.01 * y.abs())
    if before == "residual":
        within("residual", kw["residual"], h, half(dtype) * h.abs())
    # 8 bits, a scale per row; the residual is read again, so it is given anew
    for to, most in ((torch.int8, 127.0), (torch.float8_e4m3fn, 448.0)):
        kw = {} if before == "none" else {before: o.clone()}
        codes, scales = M.norm(x, w, dtype=to, **kw)
        assert scales.shape == (rows, 1) and codes.dtype == to
        check_codes(codes, scales, y, rel, most)


def check_codes(codes, scales, y, rel, most):
    want = y.abs().amax(-1, keepdim=True) / most
    within("scales", scales, want, (rel.amax() if isinstance(rel, torch.Tensor) else rel) * 1.01 * want + U * want)
    s = scales.double()
    value = codes.double() * s
    err = rel * 1.01 * y.abs() + 4 * U * y.abs()
    if most == 127.0:
        tol = 0.5 * s * (1 + 4 * U) + err
    else:                       # half a step of e4m3, or of its smallest numbers
        tol = torch.maximum(half(torch.float8_e4m3fn) * y.abs(), 2.0 ** -10 * s) * (1 + 8 * U) + 2 * err
    within("values", value, y, tol)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("group", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("rows,groups", [(3, 1), (1300, 5), (2, 37)])
def test_norm_groups(rows, groups, group, dtype):
    g = gen(group + rows)
    columns = group * groups
    x, z = normal(g, rows, columns).to(dtype), normal(g, rows, columns).to(dtype)
    w = (torch.rand(columns, device=DEV, generator=g) + 0.5).to(dtype)
    y, _, rel = norm_exact(x, w, None, z, 1e-5)
    for to, most in ((torch.int8, 127.0), (torch.float8_e4m3fn, 448.0)):
        codes, scales = M.norm(x, w, gate=z, dtype=to, group=group)
        assert scales.shape == (rows, groups)
        check_codes(codes.view(rows, groups, group), scales[..., None], y.view(rows, groups, group),
                    rel.view(rows, groups, group), most)


@pytest.mark.parametrize("dtype", [BF, F])
def test_norm_strided_rows_and_three_dimensions(dtype):
    g = gen(31)
    wide, out = normal(g, 4, 9, 640).to(dtype), torch.zeros(4, 9, 640, dtype=dtype, device=DEV)
    for cols in (slice(64, 320), slice(5, 70)):
        x, w = wide[..., cols], torch.ones(cols.stop - cols.start, dtype=dtype, device=DEV)
        y, _, rel = norm_exact(x, w, None, None, 1e-6)
        M.norm(x, w, eps=1e-6, out=out[..., cols])
        within("y", out[..., cols], y, (rel + half(dtype)) * 1.01 * y.abs())
        out[..., cols] = 0
        assert not bool(out.any())


def test_norm_rows_of_zeros_and_of_no_number():
    x = torch.zeros(4, 64, device=DEV)
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    x[3] = 1e-30
    w = torch.ones(64, device=DEV)
    y = M.norm(x, w, eps=0.0)
    assert bool(torch.isnan(y[0]).all())                       # 0 / 0, as the formula has it
    y = M.norm(x, w)
    assert not bool(y[0].any()) and bool(torch.isnan(y[1]).all())
    for to in (torch.int8, torch.float8_e4m3fn):
        codes, scales = M.norm(x, w, dtype=to, group=32)
        assert not bool(codes[0].float().any()) and not bool(scales[0].any())
        assert bool(torch.isnan(scales[1]).all()) and not bool(codes[1].float().any())
        v = codes[3].float() * scales[3].repeat_interleave(32)
        assert float((v - 1e-30 / 1e-5 ** 0.5).abs().max()) <= 0.07 * 1e-30 / 1e-5 ** 0.5


# ---------------------------------------------------------------- refusals with CUDA tensors
def test_refusals():
    x = torch.zeros(4, 2, 64, dtype=BF, device=DEV)
    dt, A = torch.zeros(4, 2, device=DEV), torch.zeros(2, device=DEV)
    st = torch.zeros(4, 2, 64, 64, device=DEV)
    ok = dict(state=st)
    for bad in (dict(B=x[:3]), dict(B=x.float()), dict(A=A.double()), dict(A=A[:1]), dict(dt=dt.half()), dict(dt=dt[:, :1]),
                dict(x=x.half()), dict(C=x[..., :32]), dict(state=st.half()), dict(state=st[:3]), dict(D=A.cpu()),
                dict(state=st.transpose(2, 3)), dict(out=x), dict(out=torch.zeros(4, 2, 64, device=DEV)),
                dict(x=torch.zeros(4, 2, 64, dtype=BF, device=DEV, requires_grad=True)),
                dict(x=torch.zeros(4, 2, 65, dtype=BF, device=DEV)[..., 1:])):
        kw = {**dict(x=x, dt=dt, A=A, B=x, C=x, D=None), **ok, **bad}
        with pytest.raises((ValueError, Q.QStateError)):
            M.scan_step(kw.pop("x"), kw.pop("dt"), kw.pop("A"), kw.pop("B"), kw.pop("C"), kw.pop("D"), **kw)
    with pytest.raises(ValueError):
        M.scan(x[None], dt[None], A, x[None], x[None], seq_starts=ints([0, 4]))
    with pytest.raises(ValueError):
        M.scan(x, dt, A, x, x, seq_starts=torch.tensor([0, 4], device=DEV))
    with pytest.raises(ValueError):
        M.scan(x, dt, A, x, x, initial=True)
    with pytest.raises(Q.QStateError):
        z = torch.zeros(4, 2, 32, dtype=BF, device=DEV)
        M.scan(z, dt, A, z, z)
    c = torch.zeros(4, 64, dtype=BF, device=DEV)
    w = torch.zeros(64, 4, dtype=BF, device=DEV)
    for kw in (dict(out=c), dict(state=torch.zeros(1, 2, 64, dtype=BF, device=DEV)), dict(initial=True),
               dict(bias=w[:, 0])):
        with pytest.raises(ValueError):
            M.conv(c, w, **kw)
    with pytest.raises(Q.QStateError):
        M.conv(c, torch.zeros(64, 5, dtype=BF, device=DEV))
    n = torch.zeros(64, dtype=BF, device=DEV)
    for kw in (dict(residual=c, gate=c), dict(dtype=torch.uint8), dict(group=32), dict(dtype=torch.int8, group=48),
               dict(residual=c[:2]), dict(out=c), dict(residual=c)):
        with pytest.raises(ValueError):
            M.norm(c, n, **kw)
    obj = Q.QState(1, 2, 64, 64, Q.GLA, bits=4)
    with pytest.raises(ValueError):
        M.step(obj, x[:1], dt[:1], A, x[:1], x[:1])
    with pytest.raises(ValueError):
        M.load(obj, torch.zeros(3, 64, 64, device=DEV))
    obj.close()


def test_empty_calls():
    x = torch.zeros(0, 2, 64, dtype=BF, device=DEV)
    dt, A = torch.zeros(0, 2, device=DEV), torch.ones(2, device=DEV)
    assert M.scan_step(x, dt, A, x, x, state=torch.zeros(0, 2, 64, 64, device=DEV)).shape == x.shape
    st = torch.ones(1, 2, 64, 64, device=DEV)
    M.scan(x, dt, A, x, x, state=st, initial=True)
    assert bool((st == 1).all())
    M.scan(x, dt, A, x, x, state=st)
    assert not bool(st.any())
    c, w = torch.zeros(0, 64, dtype=BF, device=DEV), torch.zeros(64, 4, dtype=BF, device=DEV)
    cs = torch.ones(1, 3, 64, dtype=BF, device=DEV)
    M.conv(c, w, state=cs, initial=True)
    assert bool((cs == 1).all())
    M.conv(c, w, state=cs)
    assert not bool(cs.any())
    assert M.norm(c, torch.zeros(64, dtype=BF, device=DEV), dtype=torch.int8)[1].shape == (0, 1)
    y = M.scan(x.view(0, 5, 2, 64), dt.view(0, 5, 2), A, x.view(0, 5, 2, 64), x.view(0, 5, 2, 64))
    assert y.shape == (0, 5, 2, 64)


# ---------------------------------------------------------------- streams and graphs
def test_another_stream():
    g = gen(40)
    x, dt, A, B, C, D, bias = selective(g, 3001, 1, 1, 128, 64, BF)
    want = M.scan(x, dt, A, B, C, D, dt_bias=bias)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for _ in range(20):                       # workspaces of the side stream, then of this one
        outs.append(M.scan(x, dt, A, B, C, D, dt_bias=bias, stream=s))
        torch.empty(4 << 20, dtype=torch.uint8, device=DEV).fill_(255)
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    with torch.cuda.stream(s):
        y = M.norm(x.view(3001, 64), torch.ones(64, dtype=BF, device=DEV))
    s.synchronize()
    assert torch.equal(y, M.norm(x.view(3001, 64), torch.ones(64, dtype=BF, device=DEV)))


def test_two_graphs_at_once():
    """Two captured scans that need workspaces, replayed side by side on new inputs."""
    g = gen(41)
    sets = [selective(gen(50 + i), 3001, 1, 1, 128, 64, BF) for i in range(2)]
    M.scan(*sets[0][:6], dt_bias=sets[0][6])
    graphs, outs, states = [], [], []
    for x, dt, A, B, C, D, bias in sets:
        st = torch.zeros(1, 1, 128, 64, device=DEV)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(M.scan(x, dt, A, B, C, D, dt_bias=bias, state=st))
        graphs.append(gr)
        states.append(st)
    for x, *_ in sets:
        x.copy_(normal(g, 3001, 1, 64))
    want = [M.scan(x, dt, A, B, C, D, dt_bias=bias) for x, dt, A, B, C, D, bias in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_same_call_twice_is_the_same():
    for dtype in (BF, F):
        x, dt, A, B, C, D, bias = selective(gen(60), 2000, 3, 1, 128, 128, dtype)
        a, b = (M.scan(x, dt, A, B, C, D, dt_bias=bias) for _ in range(2))
        assert torch.equal(a, b)


# ---------------------------------------------------------------- a layer's run
class Mixer:
    """A Mamba2 mixer with its state, from the operators of this package."""

    def __init__(self, g, model, heads, groups, d_k, d_v, dtype):
        self.H, self.G, self.N, self.P = heads, groups, d_k, d_v
        inner, self.ch = heads * d_v, heads * d_v + 2 * groups * d_k
        r = lambda *s: (normal(g, *s) / s[0] ** 0.5).to(dtype)  # noqa: E731
        self.win, self.wout = r(model, inner + self.ch + heads), r(inner, model)
        self.conv_w, self.conv_b = (normal(g, self.ch, 4) / 2).to(dtype), (normal(g, self.ch) / 8).to(dtype)
        self.pre, self.post = torch.ones(model, dtype=dtype, device=DEV), torch.ones(inner, dtype=dtype, device=DEV)
        _, _, self.A, _, _, self.D, self.bias = selective(g, 1, heads, groups, d_k, d_v, dtype)

    def split(self, u):
        inner = self.H * self.P
        z, mixed, dt = (u @ self.win).split([inner, self.ch, self.H], -1)
        return z, mixed, dt

    def parts(self, c):
        x, B, C = c.split([self.H * self.P, self.G * self.N, self.G * self.N], -1)
        return x.unflatten(-1, (self.H, self.P)), B.unflatten(-1, (self.G, self.N)), C.unflatten(-1, (self.G, self.N))

    def prompt(self, x, residual, starts, conv_state, state):
        u = M.norm(x, self.pre, residual=residual)
        z, mixed, dt = self.split(u)
        c = M.conv(mixed, self.conv_w, self.conv_b, state=conv_state, seq_starts=starts)
        v, B, C = self.parts(c)
        y = M.scan(v, dt, self.A, B, C, self.D, dt_bias=self.bias, state=state, seq_starts=starts)
        return M.norm(y.flatten(-2), self.post, gate=z) @ self.wout

    def token(self, x, residual, conv_state, state):
        u = M.norm(x, self.pre, residual=residual)
        z, mixed, dt = self.split(u)
        v, B, C = self.parts(M.conv_step(mixed, self.conv_w, self.conv_b, state=conv_state))
        if isinstance(state, Q.QState):
            y = M.step(state, v, dt, self.A, B, C, self.D, dt_bias=self.bias)
        else:
            y = M.scan_step(v, dt, self.A, B, C, self.D, dt_bias=self.bias, state=state)
        return M.norm(y.flatten(-2), self.post, gate=z) @ self.wout


@pytest.mark.parametrize("dtype", [F, BF])
def test_prompt_then_tokens_as_one_prompt(dtype):
    """Prompts of unequal lengths, then tokens one by one: what the layer gives for
    the whole sequences at once, on float32 states and, within their step, on
    8-bit ones that the prompt's states were loaded into."""
    g = gen(70)
    lens, extra = [130, 1, 57], 6
    layer = Mixer(g, 192, 4, 2, 64, 64, dtype)
    n = len(lens)
    full = [normal(g, k + extra, 192).to(dtype) for k in lens]
    starts = lambda ks: ints([sum(ks[:i]) for i in range(len(ks) + 1)])  # noqa: E731
    zeros = lambda t: torch.zeros_like(t)  # noqa: E731

    def states():
        return (torch.zeros(n, 3, layer.ch, dtype=dtype, device=DEV), torch.zeros(n, 4, 64, 64, device=DEV))

    whole = torch.cat(full)
    conv_w, st_w = states()
    want = layer.prompt(whole, zeros(whole), starts([k + extra for k in lens]), conv_w, st_w)
    want = want.split([k + extra for k in lens])
    head = torch.cat([f[:k] for f, k in zip(full, lens)])
    conv_s, st = states()
    got = layer.prompt(head, zeros(head), starts(lens), conv_s, st).split(lens)
    tol = 1e-4 if dtype == F else 3e-2                 # sums in another order, through two products
    scale = float(torch.cat(want).abs().max())
    for w, o, k in zip(want, got, lens):
        assert float((w[:k] - o).abs().max()) <= tol * scale
    obj = Q.QState(n, 4, 64, 64, Q.MAMBA2, bits=8, group=64)
    M.load(obj, st)
    conv_q = conv_s.clone()
    for t in range(extra):
        x = torch.stack([f[k + t] for f, k in zip(full, lens)])
        w = torch.stack([o[k + t] for o, k in zip(want, lens)])
        y = layer.token(x, zeros(x), conv_s, st)
        assert float((w - y).abs().max()) <= tol * scale, t
        q = layer.token(x, zeros(x), conv_q, obj)
        # 8-bit states: half a step of 1/127 of each group's maximum a token
        assert rel2(q, w) <= 0.01 * (t + 1) + tol, t
    assert torch.equal(conv_s, conv_q) and rel2(st, st_w) <= (1e-5 if dtype == F else 1e-2)
    if dtype == F:
        assert rel2(conv_s, conv_w) <= 1e-5
    obj.close()


def test_a_token_captured_and_replayed():
    """The decode step of a layer in one graph, on a low-bit state: replays move the
    states on as the calls do."""
    g = gen(71)
    layer = Mixer(g, 192, 4, 1, 64, 64, BF)
    x = normal(g, 5, 192).to(BF)
    runs = []
    for captured in (False, True):
        obj = Q.QState(5, 4, 64, 64, Q.MAMBA2, bits=4, group=32)
        conv = torch.zeros(5, 3, layer.ch, dtype=BF, device=DEV)
        res = torch.zeros_like(x)
        layer.token(x, res, conv, obj)
        if captured:
            torch.cuda.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                y = layer.token(x, res, conv, obj)
            for _ in range(3):
                gr.replay()
        else:
            for _ in range(3):
                y = layer.token(x, res, conv, obj)
        torch.cuda.synchronize()
        runs.append((y.clone(), conv, res, obj.dequant()))
        obj.close()
    for a, b in zip(*runs):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- wider calls
@pytest.mark.parametrize("dtype", [BF, F])
def test_scan_many_sequences_cut_unevenly(dtype):
    """More sequences than a warp counts at once, one of them long enough to be cut."""
    g = gen(90)
    lens = [3, 0, 17, 4000, 1] + [5 + i % 9 for i in range(72)]
    starts = [sum(lens[:i]) for i in range(len(lens) + 1)]
    n, T = len(lens), starts[-1]
    x, dt, A, B, C, D, bias = selective(g, T, 1, 1, 64, 64, dtype)
    st = normal(g, n, 1, 64, 64)
    want = scan_exact(x, dt, A, B, C, D, bias, True, st, starts)
    y = M.scan(x, dt, A, B, C, D, dt_bias=bias, state=st, initial=True, seq_starts=ints(starts))
    check_scan(y, st, want, dtype)


@pytest.mark.parametrize("dtype", [BF, F])
def test_scan_equal_sequences_cut(dtype):
    g = gen(91)
    n, L = 3, 1900
    x, dt, A, B, C, D, bias = selective(g, n * L, 2, 1, 128, 64, dtype)
    st = normal(g, n, 2, 128, 64)
    want = scan_exact(x, dt, A, B, C, D, bias, True, st, [0, L, 2 * L, 3 * L])
    by = [t.view(n, L, *t.shape[1:]) for t in (x, dt, B, C)]
    y = M.scan(by[0], by[1], A, by[2], by[3], D, dt_bias=bias, state=st, initial=True)
    check_scan(y.view(n * L, 2, 64), st, want, dtype)


@pytest.mark.parametrize("dtype", [BF, F])
def test_outputs_at_any_alignment(dtype):
    """Outputs that are views at odd columns of wider buffers, the columns beside
    them left as they were."""
    g = gen(92)
    T, H, N, P = 200, 2, 64, 64
    x, dt, A, B, C, D, bias = selective(g, T, H, 1, N, P, dtype)
    st = normal(g, T, H, N, P)
    for off in (1, 8, 16):
        wide = torch.full((T, 160), 3.0, dtype=dtype, device=DEV)
        out = wide[:, off:off + H * P].unflatten(-1, (H, P))
        assert torch.equal(M.scan(x, dt, A, B, C, D, dt_bias=bias, out=out), M.scan(x, dt, A, B, C, D, dt_bias=bias))
        assert bool((wide[:, :off] == 3).all()) and bool((wide[:, off + H * P:] == 3).all())
        M.scan_step(x, dt, A, B, C, D, dt_bias=bias, state=st.clone(), out=out)
        assert torch.equal(out, M.scan_step(x, dt, A, B, C, D, dt_bias=bias, state=st.clone()))
        u, w = normal(g, 9, 64).to(dtype), torch.ones(64, dtype=dtype, device=DEV)
        for to in (torch.int8, torch.float8_e4m3fn):
            codes = torch.zeros(9, 100, dtype=torch.uint8, device=DEV).view(to)
            M.norm(u, w, dtype=to, group=16, out=codes[:, off:off + 64])
            assert torch.equal(codes[:, off:off + 64].float(), M.norm(u, w, dtype=to, group=16)[0].float())
            codes[:, off:off + 64] = 0
            assert not bool(codes.float().any())


def test_offsets_past_32_bits():
    """Rows that lie further apart than 2^31 elements in all."""
    T, pitch = 70000, 32768
    wide = torch.empty(T, pitch, dtype=BF, device=DEV)               # 4.6 GB
    g = gen(93)
    x, dt, A, B, C, D, bias = selective(g, T, 1, 1, 64, 64, BF)
    cols = [wide[:, 64 * i:64 * i + 64] for i in range(4)]
    for c, t in zip(cols, (x, B, C)):
        c.copy_(t.view(T, 64))
    xv, Bv, Cv = (c.unflatten(-1, (1, 64)) for c in cols[:3])
    out = cols[3].unflatten(-1, (1, 64))
    M.scan(xv, dt, A, Bv, Cv, D, dt_bias=bias, out=out)
    assert torch.equal(out, M.scan(x, dt, A, B, C, D, dt_bias=bias))
    M.scan_step(xv, dt, A, Bv, Cv, D, dt_bias=bias, state=torch.zeros(T, 1, 64, 64, device=DEV), out=out)
    assert torch.equal(out, M.scan_step(x, dt, A, B, C, D, dt_bias=bias, state=torch.zeros(T, 1, 64, 64, device=DEV)))
    w = normal(g, 64, 4).to(BF)
    M.conv(cols[0], w, out=cols[3])
    assert torch.equal(cols[3], M.conv(x.view(T, 64), w))
    M.norm(cols[0], torch.ones(64, dtype=BF, device=DEV), gate=cols[1], out=cols[3])
    assert torch.equal(cols[3], M.norm(x.view(T, 64), torch.ones(64, dtype=BF, device=DEV), gate=B.view(T, 64)))


def test_scans_and_products_side_by_side():
    """Full scans on two streams beside matrix products on a third, which use the
    same tensor memory: all end, with the results they have alone."""
    sets = [selective(gen(94 + i), 2000, 32, 1, 128, 64, BF) for i in range(2)]
    a = normal(gen(96), 4096, 4096).to(BF)
    want = [M.scan(x, dt, A, B, C, D, dt_bias=bias) for x, dt, A, B, C, D, bias in sets]
    product = a @ a
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(6):
        for (x, dt, A, B, C, D, bias), s in zip(sets, streams):
            outs.append(M.scan(x, dt, A, B, C, D, dt_bias=bias, stream=s))
        with torch.cuda.stream(streams[2]):
            p = a @ a
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])
    assert torch.equal(p, product)


def test_conv_step_captured_and_replayed():
    """Captured once and replayed: the states move on each time."""
    g = gen(97)
    x, w = normal(g, 4, 64).to(BF), normal(g, 64, 4).to(BF)
    a = torch.zeros(4, 3, 64, dtype=BF, device=DEV)
    b = a.clone()
    M.conv_step(x, w, state=a)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y = M.conv_step(x, w, state=a)
    gr.replay()
    gr.replay()
    for _ in range(3):
        want = M.conv_step(x, w, state=b)
    assert torch.equal(y, want) and torch.equal(a, b)


# ---------------------------------------------------------------- the compiled calls
def test_usual_calls_are_the_python_ones(monkeypatch):
    """Each operator's usual call is answered by the compiled module, and with it out
    of the way the Python checks give the same bits."""
    g = gen(98)
    x, dt, A, B, C, D, bias = selective(g, 150, 4, 2, 64, 128, BF, view=True)
    st = normal(g, 150, 4, 64, 128)
    one, cs = normal(g, 1, 4, 64, 128), normal(g, 2, 3, 64).to(BF)
    u, w = normal(g, 2, 64).to(BF), normal(g, 64, 4).to(BF)
    by = lambda t: t.view(3, 50, *t.shape[1:])  # noqa: E731
    calls = {
        "scan_step": lambda: [M.scan_step(x, dt, A, B, C, D, dt_bias=bias, state=(s := st.clone())), s],
        "scan": lambda: [M.scan(x, dt, A, B, C, D, dt_bias=bias, state=(s := one.clone()), initial=True), s,
                         M.scan(x, dt, A, B, C, seq_starts=ints([0, 20, 150])),
                         M.scan(by(x.contiguous()), by(dt), A, by(B.contiguous()), by(C.contiguous()), softplus=False)],
        "conv_step": lambda: [M.conv_step(u, w, w[:, 0].contiguous(), state=(s := cs.clone())), s],
        "conv": lambda: [M.conv(x.flatten(1), w.repeat(8, 1), seq_starts=ints([0, 20, 150])),
                         M.conv(u[None], w, state=(s := cs[:1].clone()), initial=True, activation=False), s],
        "norm": lambda: [*M.norm(u, w[:, 0].contiguous(), gate=u, dtype=torch.int8, group=16),
                         M.norm(x.flatten(1), torch.ones(512, dtype=BF, device=DEV)),
                         M.norm(u, w[:, 0].contiguous(), residual=(r := u.clone()), eps=1e-3), r],
    }
    M.norm(u, w[:, 0].contiguous())
    import types
    names = ("conv", "conv_step", "scan", "scan_step", "norm")
    real = M._usual
    for name, call in calls.items():
        seen = []

        def spy(*a, _f=getattr(real, name)):
            seen.append(_f(*a))
            return seen[-1]
        monkeypatch.setattr(M, "_usual", types.SimpleNamespace(**{n: spy if n == name else getattr(real, n) for n in names}))
        got = call()
        assert seen and all(s is not None for s in seen), name
        monkeypatch.setattr(M, "_usual", types.SimpleNamespace(**{n: lambda *a: None for n in names}))
        for a, b in zip(got, call()):
            assert a.dtype == b.dtype and a.shape == b.shape, name
            a, b = a.float(), b.float()         # (time steps below zero grow until they overflow)
            assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num()), name
        monkeypatch.setattr(M, "_usual", real)


def test_compiled_calls_leave_the_rest_to_python():
    u = M._usual
    x = torch.zeros(4, 2, 64, dtype=BF, device=DEV)
    dt, A = torch.zeros(4, 2, device=DEV), torch.zeros(2, device=DEV)
    st = torch.zeros(4, 2, 64, 64, device=DEV)
    good = [x, dt, A, x, x, None, None, st, True]
    assert u.scan_step(*good) is not None
    for i, bad in ((0, None), (0, 3), (0, x.cpu()), (0, x.float()), (0, x.half()), (0, x[:3]), (0, x.transpose(0, 1)),
                   (0, torch.zeros(4, 2, 72, dtype=BF, device=DEV)[..., 1:65]), (1, dt[:, :1]), (1, dt.double()),
                   (2, A.double()), (2, None), (2, A[:1]), (3, x[..., :32]), (4, x[:, :1]), (5, A.cpu()), (6, dt[0, :1]),
                   (7, None), (7, st[:3]), (7, st.double()), (7, st.transpose(2, 3)),
                   (0, torch.zeros(4, 2, 64, dtype=BF, device=DEV, requires_grad=True))):
        assert u.scan_step(*good[:i], bad, *good[i + 1:]) is None, i
    assert u.scan_step(*good[:8]) is None and u.scan_step() is None
    with torch.no_grad():
        assert u.scan_step(torch.zeros(4, 2, 64, dtype=BF, device=DEV, requires_grad=True), *good[1:]) is not None
    # an output that would lie in an input: the state inside x
    both = torch.zeros(4 * 2 * 64 * 64, device=DEV)
    assert u.scan_step(both[:512].view(4, 2, 64), dt, A, both[:512].view(4, 2, 64), both[512:1024].view(4, 2, 64), None,
                       None, both.view(4, 2, 64, 64), True) is None
    c, w = torch.zeros(4, 64, dtype=BF, device=DEV), torch.zeros(64, 4, dtype=BF, device=DEV)
    s = torch.zeros(4, 3, 64, dtype=BF, device=DEV)
    assert u.conv_step(c, w, None, s, True) is not None
    for a in ((c, w[:, :3], None, s, True), (c, w, w[:, 0], s, True), (c, w, None, s[:3], True), (c, w, None, None, True),
              (c, w.float(), None, s, True), (c[:, :32], w, None, s, True)):
        assert u.conv_step(*a) is None
    assert u.conv(c, w, None, None, True, True, None) is None                       # nothing to continue from
    assert u.conv(c, w, None, None, True, False, torch.tensor([0, 4])) is None       # starts on the host
    n = torch.zeros(64, dtype=BF, device=DEV)
    for a in ((c, n, c, 1, 1e-5, 0, 0), (c, n, c[:2], 2, 1e-5, 0, 0), (c, n, None, 0, 1e-5, 1, 48),
              (c, n[:32], None, 0, 1e-5, 0, 0), (c, n, None, 0, "a", 0, 0), (c, n, None, 0, -1.0, 0, 0)):
        assert u.norm(*a) is None
