"""Plain 64-bit references of the attention operators, with bounds on how far
an evaluation in the documented precision may be from them.

With u = 2^-24 every fp32 operation adds u times the magnitude of its result;
sums are bounded by the sums of magnitudes, a sum of n terms by n u of them
(twice that on the tensor cores, which may cut instead of rounding), ex2.approx
and rsqrt by 4 u.  A result rounded to bf16 is off by at most 2^-8 of its
value, to fp16 by 2^-11, to e4m3 by 2^-4, or 2^-10 where it is below 2^-6.
"""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


def norm_rope(x, weight, eps, positions, inv_freq, axes=None, interleaved=False):
    """(y, bound before the last rounding) of x [T, H, D]: positions [T] or
    [axes, T]."""
    x = x.double()
    T, H, D = x.shape
    y, rel = x, 0.0
    if weight is not None:
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + eps) * weight.double()
        # the sum's D u (half of it through the root), the root, two products
        rel = (D / 2 + 8) * U
    err = rel * y.abs()
    if inv_freq is None:
        return y, err
    half = inv_freq.shape[0]
    p = positions.double()
    p = p[None].expand(half, T) if axes is None else p[torch.tensor(axes, device=p.device)]
    angle = p.t() * inv_freq.double()
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    first = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    a, b = y[..., first], y[..., second]
    ea, eb = err[..., first], err[..., second]
    # The angle: 2^-25 half turns of rounding (1.6 u), its turn's fraction and
    # this reference's own product, each 2^-53 of the angle; sine and cosine two
    # ulp; a product and a sum.
    turn = (1.6 * U + angle.abs()[:, None] * 2.0 ** -51) + 6 * U
    mag = a.abs() + b.abs() + ea + eb
    y, err = y.clone(), err.clone()
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    err[..., first] = err[..., second] = ea + eb + mag * turn
    return y, err


def rounded(y, err, dtype):
    """The bound with the rounding to `dtype`."""
    step = HALF_STEP[dtype] * (y.abs() + err)
    if dtype == torch.float8_e4m3fn:
        step = step.clamp(min=2.0 ** -10)
    return err + step


def places(cu, lens, table, page_size, pages, tokens):
    """[(token, page, slot, index)] of the tokens that are stored, and the
    index of every token that belongs to a sequence."""
    stored, index = [], {}
    width = len(table[0]) if table else 0
    for n in range(len(lens)):
        length = min(max(lens[n], 0), width * page_size)
        for t in range(cu[n], cu[n + 1]):
            j = length - (cu[n + 1] - t)
            index[t] = j
            if j >= 0 and 0 <= table[n][j // page_size] < pages:
                stored.append((t, table[n][j // page_size], j % page_size, j))
    return stored, index


def attention(q, k_cache, v_cache, table, lens, scale, gate=None, k_scale=None, v_scale=None):
    """(out, bound before the last rounding, lse, its bound) of q [N, L, Hq, D];
    table and lens as lists."""
    N, L, Hq, D = q.shape
    S, Hkv = k_cache.shape[1:3]
    G = Hq // Hkv
    dev = q.device
    small = q.dtype != torch.float32  # weights rounded to 16 bits
    eight = k_scale is not None
    out = torch.zeros(N, L, Hq, D, dtype=torch.float64, device=dev)
    err = torch.zeros_like(out)
    lse = torch.full((N, L, Hq), -torch.inf, dtype=torch.float64, device=dev)
    lse_err = torch.zeros_like(lse)
    for n in range(N):
        length = min(max(lens[n], 0), len(table[n]) * S)
        if length == 0:
            continue
        held = table[n][:-(-length // S)]
        if any(not 0 <= p < k_cache.shape[0] for p in held):
            out[n] = lse[n] = torch.nan
            continue
        held = torch.tensor(held, device=dev)

        def rows(cache, by):
            x = cache.view(torch.uint8)[held].view(cache.dtype) if eight else cache[held]
            x = x.flatten(0, 1)[:length].double().transpose(0, 1)  # [Hkv, tokens, D]
            return x if by is None else x * by.double()[:, None, None]
        k, v = rows(k_cache, k_scale), rows(v_cache, v_scale)
        for t in range(L):
            sees = length - L + 1 + t
            if sees <= 0:
                continue
            x = q[n, t].double().view(Hkv, G, D)
            ks, vs = k[:, :sees], v[:, :sees]
            s = scale * x @ ks.transpose(1, 2)                       # [Hkv, G, sees]
            mag = abs(scale) * x.abs() @ ks.abs().transpose(1, 2)
            es = (2 * D + 8) * U * mag
            if eight:  # queries as 16 bits beside their largest: 2^-24 of it
                es = es + 2.0 ** -24 * abs(scale) * x.abs().amax(-1, keepdim=True) * \
                    ks.abs().sum(-1)[:, None]
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(torch.isfinite(m), m, 0.0))
            l = p.sum(-1, keepdim=True)
            l = torch.where(m == -torch.inf, 0.0, l)
            # A weight: its score's error, the exponent's roundings, ex2, a
            # factor per eight tokens; then the sums of `sees` terms.
            rel = (es + 6 * U * (s.abs() + m.abs())).amax(-1, keepdim=True) + \
                (8 + 3 * sees) * U
            y = (p @ vs) / l
            weighted = (p @ vs.abs()) / l
            e = 2 * rel * weighted
            if small:  # weights as bf16, or as fp16 with 2^-24 the smallest
                e = e + 2.0 ** -8 * weighted + 2.0 ** -24 / l * vs.abs().sum(1)[:, None]
            empty = (l == 0).expand_as(y)
            y, e = torch.where(empty, 0.0, y), torch.where(empty, 0.0, e)
            if gate is not None:
                g = gate[n, t].double().view(Hkv, G, D)
                f = torch.sigmoid(g)
                e = e * f + (10 + 2 * g.abs()) * U * y.abs() * f
                y = y * f
            out[n, t], err[n, t] = y.reshape(Hq, D), e.reshape(Hq, D)
            z = torch.log(l) + m
            lse[n, t] = torch.where(l == 0, -torch.inf, z).reshape(Hq)
            lse_err[n, t] = (rel + 4 * U * (z.abs() + m.abs())).reshape(Hq)
    return out, err, lse, lse_err
