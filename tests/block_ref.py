"""Plain 64-bit references of the block operators, token by token, with bounds
on how far an fp32 evaluation rounded once at its end may be from them.

The bounds are running error analyses: with u = 2^-24, every fp32 operation
adds u times the magnitude of its result, ex2.approx adds two ulp (4 u) and
an exponent's rounding |exponent| u; the magnitudes are those of the same
sums with absolute values.  `u_out` is the output type's own half ulp.
"""
import numpy as np

U = 2.0 ** -24
U_BF16 = 2.0 ** -8  # two half ulps of bf16: the bound's result may round the other way


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def silu(v):
    return v * sigmoid(v)


def silu_err(v, ev):
    """Bound on silu's error at v with an error ev in v: the slope is below
    1.1; e^-v carries 2 |v| u of its exponent, sums and reciprocal 10 u."""
    return 1.1 * ev + np.abs(silu(v)) * (2.0 * np.abs(v) + 10.0) * U


def conv(x, w, cu, bias=None, init=None, act=None, u_out=U):
    """(out, bound, final state)."""
    T, C = x.shape
    K, N = w.shape[1], len(cu) - 1
    out, err = np.zeros((T, C)), np.zeros((T, C))
    fin = np.zeros((N, K - 1, C))
    for n in range(N):
        past = np.zeros((K - 1, C)) if init is None else init[n]
        seen = np.concatenate([past, x[cu[n]:cu[n + 1]]])
        fin[n] = seen[len(seen) - (K - 1):]
        for i in range(cu[n + 1] - cu[n]):
            y = np.zeros(C) if bias is None else bias.copy()
            mag = np.abs(y)
            for j in range(K):
                y = y + w[:, j] * seen[i + j]
                mag = mag + np.abs(w[:, j] * seen[i + j])
            e = (K + 1) * U * mag
            if act == "silu":
                e, y = silu_err(y, e), silu(y)
            out[cu[n] + i], err[cu[n] + i] = y, e + u_out * (np.abs(y) + e)
    return out, err, fin


def scan(x, dt, A, B, C, cu, D=None, z=None, dt_bias=None, softplus=False, init=None, u_out=U):
    """(out, bound, final state, its bound).  B, C: [T, G, S]."""
    T, d = x.shape
    G, S = B.shape[1:]
    N = len(cu) - 1
    out, err = np.zeros((T, d)), np.zeros((T, d))
    fin, fin_err = np.zeros((N, d, S)), np.zeros((N, d, S))
    Bc, Cc = np.repeat(B, d // G, axis=1), np.repeat(C, d // G, axis=1)
    for n in range(N):
        h = np.zeros((d, S)) if init is None else init[n].copy()
        mag, e = np.abs(h), np.zeros((d, S))
        # Windows joined by the exponential of a sum of up to L steps: X e^-X
        # < 0.4 times the sum's L u.
        joined = 0.4 * (cu[n + 1] - cu[n]) * U
        for t in range(cu[n], cu[n + 1]):
            v = dt[t] + (0.0 if dt_bias is None else dt_bias)
            s = np.logaddexp(0.0, v) if softplus else v
            rs = ((2.0 * np.abs(v) + 10.0) * U if softplus else 2.0 * U) * np.ones(d)
            arg = s[:, None] * A
            a = np.exp(arg)
            add = (s * x[t])[:, None] * Bc[t]
            ra = np.abs(arg) * (rs[:, None] + 4.0 * U) + 6.0 * U
            e = a * e + a * mag * ra + np.abs(add) * (rs[:, None] + 3.0 * U)
            h = a * h + add
            mag = a * mag + np.abs(add)
            e = e + 2.0 * U * mag
            terms = np.abs(Cc[t]) * (mag + e)
            y = (Cc[t] * h).sum(1)
            ey = (np.abs(Cc[t]) * (e + joined * mag)).sum(1) + (S + 3) * U * terms.sum(1)
            if D is not None:
                y = y + D * x[t]
                ey = ey + 2.0 * U * (np.abs(D * x[t]) + np.abs(y))
            if z is not None:
                gate = silu(z[t])
                ey = ey * np.abs(gate) + np.abs(y) * (silu_err(z[t], 0.0) + U * np.abs(gate))
                y = y * gate
            out[t], err[t] = y, ey + u_out * (np.abs(y) + ey)
        fin[n], fin_err[n] = h, e + joined * mag
    return out, err, fin, fin_err


def norm(y, weight=None, gate=None, residual=None, next_weight=None, act="silu", gate_first=False,
         scale=1.0, eps=1e-6, u_out=U, u_next=U):
    """(out, bound, next, its bound).  A lane sums up to 32 squares, the lanes
    join in at most ten steps: relative 48 u in the mean, half in its root."""
    g, eg = np.ones_like(y), np.zeros_like(y)
    if gate is not None:
        g = {"silu": silu, "sigmoid": sigmoid, None: lambda v: v}[act](gate)
        eg = np.abs(g) * (0.0 if act is None else 1.0) * (2.0 * np.abs(gate) + 10.0) * U
    m, em = y * g, np.abs(y) * eg + U * np.abs(y * g)
    f, ef = 1.0, 0.0
    if weight is not None:
        v, ev = (m, em) if gate_first else (y, np.zeros_like(y))
        rms = np.sqrt((v * v).mean(1, keepdims=True) + eps)
        f = weight / rms
        ef = np.abs(f) * (np.sqrt((ev * ev).mean(1, keepdims=True)) / rms + 40.0 * U)
    em = np.abs(scale) * (em * np.abs(f) + (np.abs(m) + em) * (ef + 3.0 * U * np.abs(f)))
    m = scale * m * f
    out = m if residual is None else m + residual
    err = em + U * np.abs(out)
    nxt = nerr = None
    if next_weight is not None:
        rms = np.sqrt((out * out).mean(1, keepdims=True) + eps)
        nxt = next_weight * out / rms
        rel = np.sqrt((err * err).mean(1, keepdims=True)) / rms + 40.0 * U
        nerr = np.abs(next_weight) / rms * err + np.abs(nxt) * (rel + 3.0 * U)
        nerr = nerr + u_next * (np.abs(nxt) + nerr)
    return out, err + u_out * (np.abs(out) + err), nxt, nerr
