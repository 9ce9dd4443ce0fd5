"""The mixer operators around a recurrent state: what is timed, on which sizes.

A Mamba2 layer runs, around the recurrent state that this package keeps in low-bit
codes: a short causal convolution over its channels, the selective scan of a prompt
(or the selective step of one token), the handover of the prompt's float32 state into
the low-bit object, and a root-mean-square norm whose output may be held in 8 bits.
Each case below is one call of one of them, in the form that the prompt or the
single token uses.

  conv        y_t = act(bias + sum_k w_k x_{t-W+1+k}), per channel; the last W-1 rows
              of each sequence are its state
  conv_step   the same for one token of each sequence, the state moved in place
  scan        S_t = exp(dt_t A) S_{t-1} + dt_t B_t x_t^T,  y_t = S_t^T C_t + D x_t
  scan_step   the same for one token of each sequence, the float32 state in place
  norm        h = x + residual, or x silu(gate);  y = h / rms(h) * weight, in the
              inputs' type or as 8-bit codes with a scale per row or per group
  load        a float32 state quantised into the low-bit object's codes and scales

`own` chooses between the elementary form (False) and the package's calls (True).
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"


def _type(name):
    return torch.bfloat16 if name == BF16 else torch.float32


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the benchmark's Mamba2 layer (32 heads, d_k 128, d_v 64: 2304 convolved
        # channels), eight prompts of 2048 tokens in one batch
        dict(name="conv prompt", op="conv", type=BF16, sequences=8, tokens=16384, ragged=False, channels=2304,
             width=4, initial=False, split=0),
        # the same layer decoding one token of 64 sequences
        dict(name="conv token", op="conv_step", type=BF16, sequences=64, channels=2304, width=4),
        # the benchmark's Mamba2 layer on eight prompts of 2048 tokens: the largest case
        dict(name="scan prompt", op="scan", type=BF16, sequences=8, tokens=16384, ragged=False, heads=32, groups=1,
             d_k=128, d_v=64, initial=False, split=0),
        # one long prompt, continued from a state, with the 16 heads of 128 x 128 of the
        # benchmark's larger heads: few rows and a long axis
        dict(name="scan long", op="scan", type=BF16, sequences=1, tokens=16001, ragged=False, heads=16, groups=2,
             d_k=128, d_v=128, initial=True, split=0),
        # float32 prompts of unequal lengths packed one behind the other, small heads
        dict(name="scan ragged f32", op="scan", type=F32, sequences=7, tokens=3001, ragged=True, heads=16, groups=1,
             d_k=64, d_v=64, initial=False, split=3),
        # the shortest prompt of a chat turn, where latency counts
        dict(name="scan short", op="scan", type=BF16, sequences=1, tokens=37, ragged=False, heads=32, groups=1,
             d_k=128, d_v=64, initial=True, split=0),
        # one token of 64 sequences of the benchmark's Mamba2 layer, states in float32
        dict(name="scan token", op="scan_step", type=BF16, sequences=64, heads=32, groups=1, d_k=128, d_v=64),
        # one token of one sequence: the smallest call
        dict(name="scan token one", op="scan_step", type=F32, sequences=1, heads=2, groups=1, d_k=64, d_v=64),
        # the mixer's gated norm over its 2048 value channels, a prompt batch, codes and a
        # scale per 128 columns for an 8-bit float product behind it
        dict(name="norm gated e4m3", op="norm", type=BF16, rows=16384, columns=2048, before="gate", to="e4m3", group=128),
        # the norm in front of a layer while decoding 61 sequences, int8 with a scale per row
        dict(name="norm residual int8", op="norm", type=BF16, rows=61, columns=2048, before="residual", to="int8", group=0),
        # the benchmark's Mamba2 states after their prompts, int8 with a scale per tile
        dict(name="load int8", op="load", sequences=64, heads=32, d_k=128, d_v=64, bits=8, group=0),
        # one sequence of the 16-head layer, int4 in groups of 32 columns
        dict(name="load int4", op="load", sequences=1, heads=16, d_k=128, d_v=128, bits=4, group=32),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("conv", "conv_step", "scan", "scan", "scan_step", "norm", "norm", "load"))
    kind = rng.choice((BF16, BF16, F32))
    if op == "conv":
        channels = rng.choice((_log(rng, 1, 4096), 8 * _log(rng, 1, 512)))
        tokens = _log(rng, 1, min(16384, 40_000_000 // channels))
        return dict(op=op, type=kind, **_sequences(rng, tokens), channels=channels, width=rng.choice((2, 3, 4)),
                    initial=rng.random() < 0.5)
    if op == "conv_step":
        return dict(op=op, type=kind, sequences=_log(rng, 1, 512), channels=rng.choice((_log(rng, 1, 4096), 2304)),
                    width=rng.choice((2, 3, 4)))
    if op in ("scan", "scan_step"):
        groups = rng.choice((1, 1, 2, 4))
        heads = groups * rng.choice((1, 2, 3, 5, 8)) if rng.random() < 0.6 else 32
        size = dict(heads=heads, groups=groups, d_k=rng.choice((64, 128)), d_v=rng.choice((64, 128)))
        cost = heads * size["d_k"] * size["d_v"]
        if op == "scan_step":
            return dict(op=op, type=kind, sequences=_log(rng, 1, min(256, 16_777_216 // cost)), **size)
        tokens = _log(rng, 1, min(16384, 16384 * 32 * 128 * 64 // cost // (4 if kind == F32 else 1)))
        return dict(op=op, type=kind, **_sequences(rng, tokens), **size, initial=rng.random() < 0.5)
    if op == "norm":
        group = rng.choice((0, 0, 32, 64, 128))
        columns = group * _log(rng, 1, 32) if group else rng.choice((_log(rng, 1, 8192), 8 * _log(rng, 1, 1024)))
        to = rng.choice(("int8", "e4m3")) if group else rng.choice(("same", "int8", "e4m3"))
        return dict(op=op, type=kind, rows=_log(rng, 1, min(16384, 33_000_000 // columns)), columns=columns,
                    before=rng.choice(("none", "residual", "gate")), to=to, group=group)
    bits = rng.choice((2, 4, 6, 8))
    return dict(op=op, sequences=_log(rng, 1, 64), heads=rng.choice((1, 3, 16, 32)), d_k=rng.choice((64, 128)),
                d_v=rng.choice((64, 128)), bits=bits, group=rng.choice((0, 8, 32, 64)))


def _sequences(rng, tokens):
    ragged = rng.random() < 0.6
    n = _log(rng, 1, min(32, tokens))
    return dict(sequences=n, tokens=tokens if ragged else tokens // n * n, ragged=ragged, split=rng.randrange(1000))


def _lengths(case):
    """Tokens of each sequence: equal, or cut at random places (an empty one may come of it)."""
    n, tokens = case["sequences"], case["tokens"]
    if not case["ragged"]:
        return [tokens // n] * n
    rng = random.Random(case["split"])
    cuts = [0] + sorted(rng.randint(0, tokens) for _ in range(n - 1)) + [tokens]
    return [b - a for a, b in zip(cuts, cuts[1:])]


# ---------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _uniform(g, low, high, *shape):
    return torch.rand(*shape, device="cuda", generator=g) * (high - low) + low


def _silu(x):
    return x / (1 + torch.exp(-x))


def _sequence_state(case, s):
    lengths = _lengths(case)
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    s["lengths"] = lengths
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["sequence"] = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"),
                                            torch.tensor(lengths, device="cuda"))


def _by_sequence(case, t):
    """Equal sequences come as a batch, unequal ones packed."""
    return t if case["ragged"] else t.view(case["sequences"], -1, *t.shape[1:])


def _selective(case, g, rows):
    """x, B, C as a convolution and its activation leave them (views of one buffer), raw
    time steps whose softplus runs over 0.001 to 0.1, decay rates of 1 to 16."""
    t, H, G, N, P = _type(case["type"]), case["heads"], case["groups"], case["d_k"], case["d_v"]
    mixed = _silu(_normal(g, rows, H * P + 2 * G * N)).to(t)
    step = torch.exp(_uniform(g, math.log(0.001), math.log(0.1), H))
    return dict(mixed=mixed, x=mixed[:, :H * P].view(rows, H, P), B=mixed[:, H * P:H * P + G * N].view(rows, G, N),
                C=mixed[:, H * P + G * N:].view(rows, G, N), dt=_normal(g, rows, H).to(t),
                dt_bias=torch.log(torch.expm1(step)), A=-_uniform(g, 1, 16, H), D=_uniform(g, 0.5, 1.5, H))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case=case)
    t = _type(case["type"]) if "type" in case else torch.float32
    if op in ("conv", "conv_step"):
        C, W = case["channels"], case["width"]
        if op == "conv":
            _sequence_state(case, s)
        s["x"] = _normal(g, case["tokens"] if op == "conv" else case["sequences"], C).to(t)
        s["weight"] = _uniform(g, -1, 1, C, W).div_(math.sqrt(W)).to(t)
        s["bias"] = _uniform(g, -0.5, 0.5, C).to(t)
        s["state"] = _normal(g, case["sequences"], W - 1, C).to(t)
    elif op in ("scan", "scan_step"):
        if op == "scan":
            _sequence_state(case, s)
        s.update(_selective(case, g, case["tokens"] if op == "scan" else case["sequences"]))
        s["state"] = _normal(g, case["sequences"], case["heads"], case["d_k"], case["d_v"]).mul_(0.2)
    elif op == "norm":
        shape = (case["rows"], case["columns"])
        s["x"] = _normal(g, *shape).to(t)
        s["other"] = _normal(g, *shape).to(t) if case["before"] != "none" else None
        s["weight"] = _uniform(g, 0.5, 1.5, case["columns"]).to(t)
    else:
        s["S"] = _normal(g, case["sequences"] * case["heads"], case["d_k"], case["d_v"]) * 0.2
        if own:
            s["object"] = _object(case)
    return s


def _object(case):
    """The low-bit object that a program keeps for a layer's states."""
    from bit_recurrent_state_decode_b200 import qstate as Q
    return Q.QState(case["sequences"], case["heads"], case["d_k"], case["d_v"], Q.MAMBA2, bits=case["bits"],
                    group=case["group"])


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    return _own(case, s) if own else _PLAIN[case["op"]](case, s)


def _own(case, s):
    from bit_recurrent_state_decode_b200 import qmixer
    op = case["op"]
    if op == "conv":
        y = qmixer.conv(_by_sequence(case, s["x"]), s["weight"], s["bias"], state=s["state"], initial=case["initial"],
                        seq_starts=s["starts"] if case["ragged"] else None)
        return dict(y=y.view(s["x"].shape), state=s["state"])
    if op == "conv_step":
        return dict(y=qmixer.conv_step(s["x"], s["weight"], s["bias"], state=s["state"]), state=s["state"])
    if op == "scan":
        x, dt, B, C = (_by_sequence(case, s[k]) for k in ("x", "dt", "B", "C"))
        y = qmixer.scan(x, dt, s["A"], B, C, s["D"], dt_bias=s["dt_bias"], state=s["state"], initial=case["initial"],
                        seq_starts=s["starts"] if case["ragged"] else None)
        return dict(y=y.view(s["x"].shape), state=s["state"])
    if op == "scan_step":
        y = qmixer.scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], dt_bias=s["dt_bias"], state=s["state"])
        return dict(y=y, state=s["state"])
    if op == "norm":
        to = {"same": None, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[case["to"]]
        got = qmixer.norm(s["x"], s["weight"], dtype=to, group=case["group"], **_before(case, s))
        y = got if to is None else _values(*got)
        return dict(y=y, residual=s["other"]) if case["before"] == "residual" else dict(y=y)
    qmixer.load(s["object"], s["S"])
    return dict(state=s["object"].dequant())


def _before(case, s):
    return {} if case["before"] == "none" else {case["before"]: s["other"]}


def _values(codes, scales):
    """What 8-bit codes and their scales stand for, in the activations' 16 bits."""
    rows, columns = codes.shape
    c = codes.view(rows, scales.shape[1], -1)
    c = c if c.dtype == torch.int8 else c.to(torch.bfloat16)
    return torch.mul(c, scales[..., None], out=torch.empty(c.shape, dtype=torch.bfloat16, device=c.device)).view(rows, columns)


# ---------------------------------------------------------------- the plain forms
def _plain_conv(case, s):
    x, w, W = s["x"].float(), s["weight"].float(), case["width"]
    seq, starts, n = s["sequence"], s["starts"].long(), case["sequences"]
    rows = torch.cat([s["state"].float().view(n * (W - 1), -1), x])     # histories, then tokens

    def at(seq, place):
        """The row of `rows` at a place of a sequence; places below 0 are its history."""
        return torch.where(place >= 0, starts[seq] + place + n * (W - 1), seq * (W - 1) + W - 1 + place)

    place = (torch.arange(len(x), device="cuda") - starts[seq])[:, None] + torch.arange(1 - W, 1, device="cuda")
    taps = rows[at(seq[:, None], place)]
    every = torch.arange(n, device="cuda")
    last = (starts[1:] - starts[:-1])[:, None] + torch.arange(1 - W, 0, device="cuda")
    state = rows[at(every[:, None], last)]
    if not case["initial"]:
        taps, state = taps * (place >= 0)[..., None], state * (last >= 0)[..., None]
    y = _silu((taps * w.t()).sum(1) + s["bias"].float())
    s["state"].copy_(state)
    return dict(y=y.to(s["x"].dtype), state=s["state"])


def _plain_conv_step(case, s):
    rows = torch.cat([s["state"], s["x"][:, None]], 1)
    y = _silu((rows.float() * s["weight"].float().t()).sum(1) + s["bias"].float())
    s["state"].copy_(rows[:, 1:])
    return dict(y=y.to(s["x"].dtype), state=s["state"])


def _steps(s):
    """Time steps (softplus of the raw ones) and the logarithms of the decays."""
    z = s["dt"].float() + s["dt_bias"]
    dt = torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))
    return dt, dt.double() * s["A"].double()


def _plain_scan(case, s):
    """Pieces of 64 tokens: products inside a piece, one state per piece, and the states
    carried from piece to piece by the products of their decays. A state that a sequence
    starts from stands in front of it as d_k tokens that do not decay."""
    H, G, N, P, n = case["heads"], case["groups"], case["d_k"], case["d_v"], case["sequences"]
    Q = 64
    dt, log = _steps(s)
    x, B, C, seq = s["x"].float(), s["B"].float(), s["C"].float(), s["sequence"]
    T = len(x)
    every = torch.arange(n, device="cuda")
    starts = s["starts"].long()
    front = N if case["initial"] else 0
    at = torch.arange(T, device="cuda") + (seq + 1) * front             # where each token goes
    total = -(-(T + n * front) // Q) * Q

    def place(t, rows, *shape):
        full = torch.zeros(total, *shape, dtype=t.dtype, device="cuda")
        full[rows] = t
        return full

    X, Bs, Cs, ds, ls = place(x, at, H, P), place(B, at, G, N), place(C, at, G, N), place(dt, at, H), place(log, at, H)
    ids = place(seq + 1, at)                                            # 0: no sequence
    if front:
        lead = ((starts[:-1] + every * front)[:, None] + torch.arange(N, device="cuda")).view(-1)
        X[lead] = s["state"].permute(0, 2, 1, 3).reshape(n * N, H, P)
        Bs[lead] = torch.eye(N, device="cuda").repeat(n, 1)[:, None].expand(-1, G, -1)
        ds[lead] = 1.0
        ids[lead] = (every + 1).repeat_interleave(N)
    c = torch.cumsum(ls, 0).view(-1, Q, H).permute(2, 0, 1)             # H, pieces, Q (64 bits)
    X, ds = X.view(-1, Q, H, P).permute(2, 0, 1, 3), ds.view(-1, Q, H).permute(2, 0, 1)
    Bs, Cs = (t.view(-1, Q, G, N).permute(2, 0, 1, 3).repeat_interleave(H // G, 0) for t in (Bs, Cs))
    ids = ids.view(-1, Q)

    def decay(later, earlier, keep):
        return torch.exp((later - earlier).masked_fill(~keep, -math.inf).float())

    same = (ids[:, :, None] == ids[:, None, :]) & torch.ones(Q, Q, dtype=torch.bool, device="cuda").tril()
    xd = X * ds[..., None]
    y = (Cs @ Bs.transpose(-1, -2) * decay(c[..., :, None], c[..., None, :], same)) @ xd
    end, last = c[..., -1], ids[:, -1]                                  # of each piece
    local = (Bs * decay(end[..., None], c, ids == last[:, None])[..., None]).transpose(-1, -2) @ xd
    joined = (last[:, None] == last[None, :]) & torch.ones(len(last), len(last), dtype=torch.bool, device="cuda").tril()
    carried = (decay(end[:, :, None], end[:, None, :], joined) @ local.flatten(2)).view_as(local)
    before = torch.cat([torch.zeros_like(carried[:, :1]), carried[:, :-1]], 1)      # in front of each piece
    end_b = torch.cat([torch.zeros_like(end[:, :1]), end[:, :-1]], 1)
    last_b = torch.cat([torch.zeros_like(last[:1]), last[:-1]])
    y = y + (Cs * decay(c, end_b[..., None], ids == last_b[:, None])[..., None]) @ before
    y = y.permute(1, 2, 0, 3).reshape(total, H, P)[at] + x * s["D"][:, None]
    # the state of each sequence behind its last token (none: it stays, or is zero)
    stop = starts[1:] + (every + 1) * front - 1
    some = stop >= starts[:-1] + every * front
    stop = torch.where(some, stop, 0)
    piece, off = stop // Q, stop % Q
    c_stop = c[:, piece, off]
    mine = (ids[piece] == (every + 1)[:, None]) & (torch.arange(Q, device="cuda") <= off[:, None])
    final = (Bs[:, piece] * decay(c_stop[..., None], c[:, piece], mine)[..., None]).transpose(-1, -2) @ xd[:, piece]
    final = final + before[:, piece] * decay(c_stop, end_b[:, piece], last_b[piece] == every + 1)[..., None, None]
    s["state"].copy_((final * some[None, :, None, None]).transpose(0, 1))
    return dict(y=y.to(s["x"].dtype), state=s["state"])


def _plain_scan_step(case, s):
    dt, log = _steps(s)
    k = case["heads"] // case["groups"]
    x, B, C = s["x"].float(), s["B"].float().repeat_interleave(k, 1), s["C"].float().repeat_interleave(k, 1)
    S = s["state"] * torch.exp(log.float())[..., None, None] + (B * dt[..., None])[..., None] * x[..., None, :]
    s["state"].copy_(S)
    y = (S * C[..., None]).sum(2) + x * s["D"][:, None]
    return dict(y=y.to(s["x"].dtype), state=s["state"])


def _plain_norm(case, s):
    h = s["x"].float()
    if case["before"] == "residual":
        h = h + s["other"].float()
        s["other"].copy_(h)
    elif case["before"] == "gate":
        h = h * _silu(s["other"].float())
    y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["columns"] + 1e-5) * s["weight"].float()
    if case["to"] == "same":
        y = y.to(s["x"].dtype)
    else:
        most = 127.0 if case["to"] == "int8" else 448.0
        y = y.view(case["rows"], -1, case["group"] or case["columns"])
        scale = y.abs().amax(2).double().div(most).float()
        codes = torch.where(scale[..., None] > 0, y / scale[..., None], 0.0).clamp(-most, most)
        codes = codes.round().to(torch.int8) if case["to"] == "int8" else codes.to(torch.float8_e4m3fn)
        y = _values(codes.view(case["rows"], -1), scale)
    return dict(y=y, residual=s["other"]) if case["before"] == "residual" else dict(y=y)


def _plain_load(case, s):
    most = 2.0 ** (case["bits"] - 1) - 1
    S = s["S"]
    flat = S.view(-1, case["group"]) if case["group"] else S.view(len(S), -1)
    scale = (flat.abs().amax(1).double() / most).float().half().float()
    inverse = torch.where(scale > 0, 1 / scale, 0.0)
    codes = (flat.double() * inverse.double()[:, None]).round().clamp(-most, most)     # ties are decided exactly
    return dict(state=(codes.float() * scale[:, None]).view_as(S))


_PLAIN = dict(conv=_plain_conv, conv_step=_plain_conv_step, scan=_plain_scan, scan_step=_plain_scan_step,
              norm=_plain_norm, load=_plain_load)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, size = case["op"], 2 if case.get("type") == BF16 else 4
    if op in ("conv", "conv_step"):
        rows = case["tokens"] if op == "conv" else case["sequences"]
        C, W = case["channels"], case["width"]
        history = case["sequences"] * (W - 1) * C * (2 if op == "conv_step" or case["initial"] else 1)
        return dict(bytes=size * (2 * rows * C + history + C * (W + 1)), flops=rows * C * (2 * W + 4))
    if op in ("scan", "scan_step"):
        rows = case["tokens"] if op == "scan" else case["sequences"]
        H, G, N, P = case["heads"], case["groups"], case["d_k"], case["d_v"]
        states = case["sequences"] * H * N * P * 4 * (2 if op == "scan_step" or case["initial"] else 1)
        return dict(bytes=size * rows * (2 * H * P + 2 * G * N + H) + states + 12 * H,
                    flops=rows * H * (5 * N * P + 3 * P + 10))
    if op == "norm":
        elements, to = case["rows"] * case["columns"], 1 if case["to"] != "same" else size
        scales = 0 if case["to"] == "same" else 4 * (elements // case["group"] if case["group"] else case["rows"])
        passes = {"none": 1, "gate": 2, "residual": 3}[case["before"]]
        values = 0 if case["to"] == "same" else 3 * elements             # codes read, their values written
        return dict(bytes=elements * (size * passes + to) + values + scales + size * case["columns"], flops=8 * elements)
    elements = case["sequences"] * case["heads"] * case["d_k"] * case["d_v"]
    scales = 2 * (elements // case["group"] if case["group"] else case["sequences"] * case["heads"])
    return dict(bytes=elements * (4 + 4) + 2 * (elements * case["bits"] // 8 + scales), flops=4 * elements)


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op = case["op"]
    if op in ("conv", "conv_step"):
        x, w, b, h = d["x"], d["weight"], d["bias"], d["state"]
        W, y, states, a = case["width"], [], [], 0
        for i, n in enumerate(s["lengths"] if op == "conv" else [1] * case["sequences"]):
            kept = h[i] if op == "conv_step" or case["initial"] else torch.zeros_like(h[i])
            rows = torch.cat([kept, x[a:a + n]])
            z = sum(rows[k:k + n] * w[:, k] for k in range(W)) + b
            y.append(z * torch.sigmoid(z))
            states.append(rows[n:])
            a += n
        return dict(y=torch.cat(y), state=torch.stack(states))
    if op in ("scan", "scan_step"):
        return _exact_scan(case, s, d)
    if op == "norm":
        return _exact_norm(case, d)
    most = 2.0 ** (case["bits"] - 1) - 1
    parts = d["S"].reshape(-1, case["group"] or case["d_k"] * case["d_v"])
    scale = (parts.abs().max(1, keepdim=True).values / most).float().half().double()
    code = torch.clamp(torch.round(parts * scale.reciprocal().float().double()), -most, most)
    return dict(state=torch.where(scale > 0, code * scale, torch.zeros_like(code)).view_as(d["S"]))


def _exact_scan(case, s, d):
    """The recurrence itself, token by token, all sequences at once."""
    H, G, N, P, n = case["heads"], case["groups"], case["d_k"], case["d_v"], case["sequences"]
    lengths = s["lengths"] if case["op"] == "scan" else [1] * n
    S = d["state"].clone()
    if case["op"] == "scan" and not case["initial"]:
        S.zero_()
    first = torch.tensor([sum(lengths[:i]) for i in range(n)], device="cuda")
    left = torch.tensor(lengths, device="cuda")
    dt = torch.nn.functional.softplus(d["dt"] + d["dt_bias"], threshold=700.0)
    a = torch.exp(dt * d["A"])
    y = torch.empty_like(d["x"])
    for t in range(max(lengths)):
        all_on = t < min(lengths)
        on = slice(None) if all_on else (left > t).nonzero()[:, 0]
        rows = first[on] + t
        k = d["B"][rows].view(-1, G, 1, N).expand(-1, G, H // G, N).reshape(-1, H, N)
        q = d["C"][rows].view(-1, G, 1, N).expand(-1, G, H // G, N).reshape(-1, H, N)
        v = d["x"][rows] * dt[rows][..., None]
        new = S[on].mul_(a[rows][..., None, None]) if all_on else S[on] * a[rows][..., None, None]
        new.addcmul_(k[..., None], v[..., None, :])
        if not all_on:
            S[on] = new
        y[rows] = torch.matmul(q[..., None, :], new)[..., 0, :]
    return dict(y=y + d["x"] * d["D"][:, None], state=S)


def _exact_norm(case, d):
    h = d["x"]
    if case["before"] == "residual":
        h = h + d["other"]
    elif case["before"] == "gate":
        h = h * d["other"] * torch.sigmoid(d["other"])
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-5) * d["weight"]
    if case["to"] != "same":
        most = 127.0 if case["to"] == "int8" else 448.0
        parts = y.unflatten(1, (-1, case["group"] or case["columns"]))
        scale = parts.abs().amax(-1, keepdim=True) / most
        z = parts / torch.where(scale > 0, scale, torch.ones_like(scale))
        if case["to"] == "int8":
            z = torch.round(z)
        else:       # e4m3: 3 bits behind the point, the smallest exponent is -6
            unit = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
            z = torch.round(z / unit) * unit
        y = (z * scale).flatten(1)
    # the norm is over h in 64 bits; the residual that a float type holds is its rounding
    return dict(y=y, residual=h) if case["before"] == "residual" else dict(y=y)
