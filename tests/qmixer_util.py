"""The mixer operators from their definitions in 64 bits, with the bounds their
tests allow: each value comes with a running bound of the rounding errors that
the binary32 arithmetic may make on the way.

u = 2^-24 is half a step of binary32; half(t) is half a step of an output type
(bf16 2^-8, e4m3 2^-4), relative to the value."""
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def lengths_of(starts):
    return [b - a for a, b in zip(starts, starts[1:])]


def conv_exact(x, w, b, state, starts, act):
    """y, the states behind, and a bound of |y|'s error before the output's rounding."""
    W = w.shape[1]
    x, w, state = x.double(), w.double(), state.double()
    b = torch.zeros(x.shape[1], dtype=torch.float64, device=x.device) if b is None else b.double()
    y, bound = torch.zeros_like(x), torch.zeros_like(x)
    states = state.clone()
    for i, n in enumerate(lengths_of(starts)):
        rows = torch.cat([state[i], x[starts[i]:starts[i] + n]])
        z, most = b.expand(n, -1).clone(), b.abs().expand(n, -1).clone()
        for k in range(W):
            z = z + rows[k:k + n] * w[:, k]
            most = most + (rows[k:k + n] * w[:, k]).abs()
        # W + 1 roundings of sums; silu has a slope below 1.1, its exponential and
        # division are off by at most 2 + 1.2|z| and 2 units of binary32 (2u each)
        e = (W + 1) * U * most
        s = slice(starts[i], starts[i] + n)
        if act:
            y[s] = z * torch.sigmoid(z)
            e = 1.1 * e + y[s].abs() * (8 + 2.4 * z.abs()) * U
        else:
            y[s] = z
        bound[s] = e
        states[i] = rows[n:]
    return y, states, bound


def scan_exact(x, dt, A, B, C, D, dt_bias, softplus, state, starts):
    """(y, states, bound of y, bound of the states, magnitude of y's terms): the
    recurrence token by token, and beside it the same of magnitudes and of errors.

    A state's error: what it had, decayed; of the decay, its exponential of a
    product (off by (3 + 2|dt A|) u), one or two products with others (the chunked
    form multiplies decays among themselves: 4 u a token covers it) and the sum;
    of the token's own term, up to 24 roundings of dt's softplus, its logarithm and
    its products, and the 128 u that a tensor-core sum over a chunk may lose."""
    H, P = x.shape[-2:]
    G, N = B.shape[-2:]
    f = torch.float64
    x, dt, B, C = x.to(f), dt.to(f), B.to(f), C.to(f)
    A, D = A.to(f), torch.zeros(H, dtype=f, device=x.device) if D is None else D.to(f)
    z = dt + (0 if dt_bias is None else dt_bias.to(f))
    dt = torch.nn.functional.softplus(z, threshold=700.0) if softplus else z
    B, C = B.repeat_interleave(H // G, -2), C.repeat_interleave(H // G, -2)
    a, da = torch.exp(dt * A), (dt * A).abs()
    y, by, most = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    S = state.to(f).clone()
    SM, SE = S.abs(), torch.zeros_like(S)
    lens = torch.tensor(lengths_of(starts), device=x.device)
    first = torch.tensor(starts[:-1], device=x.device)
    for t in range(int(lens.max()) if len(lens) else 0):
        on = (lens > t).nonzero()[:, 0]
        r = first[on] + t
        ar, dr = a[r][..., None, None], da[r][..., None, None]
        term = (B[r] * dt[r][..., None])[..., None] * x[r][..., None, :]
        SE[on] = ar * (SE[on] + (8 + 2 * dr) * U * SM[on]) + (152 + 2 * z[r].abs()[..., None, None]) * U * term.abs()
        S[on] = ar * S[on] + term
        SM[on] = ar * SM[on] + term.abs()
        q = C[r][..., None]
        y[r] = (q * S[on]).sum(-2) + D[:, None] * x[r]
        most[r] = (q.abs() * SM[on]).sum(-2) + (D[:, None] * x[r]).abs()
        by[r] = (q.abs() * SE[on]).sum(-2) + (N + 8) * U * most[r]
    return y, S, by, SE + 2 * U * SM, most


def norm_exact(x, w, residual, gate, eps):
    """y, h, and the relative error of y in binary32: the sum of squares (64 in a
    row, then a tree: 80 u, half of it behind the root), the gate's silu, the root,
    reciprocal and products."""
    h = x.double()
    rel = 64 * U
    if residual is not None:
        h = h + residual.double()
    if gate is not None:
        g = gate.double()
        h = h * g * torch.sigmoid(g)
        rel = rel + (10 + 2.4 * g.abs()) * U
        rel = rel.amax(-1, keepdim=True) + rel
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()
    return y, h, rel


def within(name, got, want, tol):
    """Every element inside its bound; NaN and infinities where they are wanted."""
    got = got.double()
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN elsewhere"
    d = torch.where(odd, torch.zeros_like(want), (got - want).abs())
    over = d > torch.where(odd, torch.ones_like(want), tol + torch.zeros_like(want))
    if bool(over.any()):
        i = int(over.reshape(-1).nonzero()[0])
        raise AssertionError(f"{name}: {int(over.sum())} of {over.numel()} off, first at {i}: {got.reshape(-1)[i]} "
                             f"for {want.reshape(-1)[i]}")


def rel2(got, want):
    n = float(want.double().norm())
    return float((got.double() - want.double()).norm()) / n if n else float(got.double().norm())
