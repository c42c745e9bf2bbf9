"""Cases, plain forms and 64-bit values of the layer's neighbours in a hybrid model.

The operators, with the entry points that a user calls for them:

* conv       gdn_short_conv: short causal depthwise convolution over packed
             sequences, with its window state carried in and out
* conv_step  gdn_short_conv_step: the same for one token of each sequence
* scan       gdn_selective_scan: selective state space scan over packed
             sequences, with its state carried in and out
* scan_step  gdn_selective_scan_step: the same for one token of each sequence
* norm       gdn_norm_gate_residual: the norm after a block with its gate and
             scaled residual, and the norm before the next block

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits, rounded once at the end; with ``own`` true it calls the entry points.
``exact`` evaluates the definitions step by step in 64 bits.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Largest drawn sizes, elements of each operator's largest tensor.
_MOST_CONV = 70904 * 2048
_MOST_SCAN = 20480 * 6144 * 16
_MOST_STEP = 256 * 6144 * 16
_MOST_NORM = 4000 * 48 * 128


def listed():
    return [
        # The 4000-token prompt of the layer's prefill: q, k and v of 16 key and 48
        # value heads of 128 convolved together, read from a wider projection, going
        # on from a cached prefix.
        dict(name="conv_prompt", op="conv", dtype="bf16", tokens=4000, seqs=1, channels=10240, width=4, silu=True,
             bias=False, state=True, wide=True),
        # Many short prompts, some empty or of one token, of an odd channel count in fp32.
        dict(name="conv_ragged", op="conv", dtype="f32", tokens=5003, seqs=61, channels=1023, width=3, silu=False,
             bias=True, state=False, wide=False),
        # A single user's next token: the call's latency.
        dict(name="conv_token", op="conv_step", dtype="bf16", batch=1, channels=10240, width=4, silu=True, bias=False,
             wide=True),
        # A full server's next tokens.
        dict(name="conv_batch", op="conv_step", dtype="bf16", batch=256, channels=10240, width=4, silu=True,
             bias=True, wide=True),
        # The same 4000-token prompt through a state space layer of the value heads'
        # width (48 x 128), x and z halves of one projection, resumed from a state.
        dict(name="scan_prompt", op="scan", dtype="bf16", tokens=4000, seqs=1, channels=6144, states=16, groups=1,
             gate=True, skip=True, state=True, wide=True),
        # Many short prompts, some empty or of one token, odd sizes, two groups, fp32.
        dict(name="scan_ragged", op="scan", dtype="f32", tokens=3001, seqs=37, channels=1538, states=7, groups=2,
             gate=False, skip=True, state=True, wide=False),
        # One long document.
        dict(name="scan_long", op="scan", dtype="bf16", tokens=20480, seqs=1, channels=6144, states=16, groups=1,
             gate=True, skip=True, state=False, wide=True),
        # A single user's next token: the call's latency.
        dict(name="scan_token", op="scan_step", dtype="bf16", batch=1, channels=6144, states=16, groups=1, gate=True,
             skip=True, wide=True),
        # A full server's next tokens: the states of all users read and written.
        dict(name="scan_batch", op="scan_step", dtype="bf16", batch=256, channels=6144, states=16, groups=1,
             gate=True, skip=True, wide=True),
        # One token between two blocks: the call's latency.
        dict(name="norm_token", op="norm", dtype="bf16", res="bf16", rows=1, dim=6144, weight=True, gate=False,
             act="silu", first=False, residual=True, next=True, wide=False),
        # A prompt between two blocks, the residual stream kept in fp32.
        dict(name="norm_block", op="norm", dtype="bf16", res="f32", rows=4000, dim=6144, weight=True, gate=True,
             act="sigmoid", first=False, residual=True, next=True, wide=False),
        # The gated norm of every value head's output, before the output projection.
        dict(name="norm_heads", op="norm", dtype="bf16", res="bf16", rows=4000 * 48, dim=128, weight=True, gate=True,
             act="silu", first=False, residual=False, next=False, wide=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan", "scan_step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    coin = lambda: rng.random() < 0.5  # noqa: E731
    if op == "conv":
        channels = _log(rng, 16, 10240)
        channels = channels if coin() else -(-channels // 8) * 8
        tokens = min(_log(rng, 1, 70904), _MOST_CONV // channels)
        return dict(op=op, dtype=dtype, tokens=tokens, seqs=rng.choice([1, 1, _log(rng, 1, 200)]), channels=channels,
                    width=rng.choice([2, 3, 4, 4, 4, 5, 8]), silu=coin(), bias=coin(), state=coin(), wide=coin())
    if op == "conv_step":
        channels = _log(rng, 16, 10240)
        channels = channels if coin() else -(-channels // 8) * 8
        return dict(op=op, dtype=dtype, batch=_log(rng, 1, 512), channels=channels,
                    width=rng.choice([2, 3, 4, 4, 4, 5, 8]), silu=coin(), bias=coin(), wide=coin())
    if op in ("scan", "scan_step"):
        states = rng.choice([1, 4, 5, 8, 13, 16, 16, 16, 32, 64])
        groups = rng.choice([1, 1, 1, 2, 4])
        per = _log(rng, 32, 6144) // groups + 1
        channels = groups * (per if coin() else -(-per // 8) * 8)
        case = dict(op=op, dtype=dtype, channels=channels, states=states, groups=groups, gate=coin(), skip=coin(),
                    wide=coin())
        if op == "scan_step":
            return dict(case, batch=max(1, min(_log(rng, 1, 512), _MOST_STEP // (channels * states))))
        tokens = max(1, min(_log(rng, 1, 70904), _MOST_SCAN // (channels * states)))
        return dict(case, tokens=tokens, seqs=rng.choice([1, 1, _log(rng, 1, 200)]), state=coin())
    dim = _log(rng, 32, 16384)
    dim = dim if coin() else -(-dim // 8) * 8
    weight, residual = rng.random() < 0.8, coin()
    return dict(op=op, dtype=dtype, res="f32" if dtype == "f32" or (residual and coin()) else "bf16",
                rows=max(1, min(_log(rng, 1, 200000), _MOST_NORM // dim)), dim=dim, weight=weight, gate=coin(),
                act=rng.choice(["silu", "sigmoid"]), first=coin(), residual=residual, next=coin() or not weight,
                wide=coin())


def _lengths(case):
    """The lengths of the packed sequences: spread over the logarithm, empty ones and single tokens among them."""
    tokens, seqs = case["tokens"], case["seqs"]
    if seqs == 1:
        return [tokens]
    rng = random.Random(tokens * 1000003 + seqs)
    shares = [0.0 if rng.random() < 0.1 else math.exp(rng.uniform(0.0, 4.0)) for _ in range(seqs)]
    shares[rng.randrange(seqs)] += 1.0
    total, lens, used, seen = sum(shares), [], 0, 0.0
    for s in shares:
        seen += s
        end = int(round(tokens * seen / total))
        lens.append(end - used)
        used = end
    return lens


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, f32 = _DTYPES[case["dtype"]], torch.float32

    def normal(*shape, dtype=dt, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    def uniform(*shape, low=0.0, high=1.0):
        return torch.rand(*shape, generator=gen, device="cuda") * (high - low) + low

    def columns(rows, *widths):
        """[rows, w] for each w: slices of the columns of one projection, or tensors of their own."""
        if not case["wide"]:
            return [normal(rows, w) for w in widths]
        return list(normal(rows, sum(widths) + 8).split([*widths, 8], dim=1))[:-1]

    s = {"case": case}
    op = case["op"]
    if op in ("conv", "scan"):
        lens = _lengths(case)
        s["longest"] = max(lens)
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        rows, seqs = case["tokens"], case["seqs"]
    elif op != "norm":
        rows = seqs = case["batch"]
    if op in ("conv", "conv_step"):
        c, k = case["channels"], case["width"]
        s["x"] = columns(rows, c, 64)[0]
        s["weight"] = normal(c, k, dtype=f32, std=k ** -0.5)
        s["bias"] = normal(c, dtype=f32, std=0.1) if case["bias"] else None
        s["state"] = normal(seqs, k - 1, c) if op == "conv_step" or case["state"] else None
        s["act"] = "silu" if case["silu"] else None
    elif op in ("scan", "scan_step"):
        d, n, g = case["channels"], case["states"], case["groups"]
        s["x"], s["z"] = columns(rows, d, d)
        s["z"] = s["z"] if case["gate"] else None
        low, b, c = columns(rows, 8, g * n, g * n)
        s["B"], s["C"] = b.unflatten(1, (g, n)), c.unflatten(1, (g, n))
        s["dt"] = normal(rows, d, std=0.5)
        # Steps log-uniform over [0.001, 0.1] through the softplus; decay rates 1 .. n.
        step = torch.exp(uniform(d, low=math.log(1e-3), high=math.log(1e-1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A"] = -torch.arange(1, n + 1, device="cuda", dtype=f32) * uniform(d, n, low=0.8, high=1.25)
        s["D"] = normal(d, dtype=f32, std=0.2, mean=1.0) if case["skip"] else None
        s["state"] = normal(seqs, d, n, dtype=f32, std=0.3) if op == "scan_step" or case["state"] else None
    else:
        r, d = case["rows"], case["dim"]
        res = _DTYPES[case["res"]]
        s["y"] = columns(r, d, 16)[0]
        s["weight"] = normal(d, dtype=f32, std=0.2, mean=1.0) if case["weight"] else None
        s["gate"] = columns(r, d, 16)[0] if case["gate"] else None
        s["residual"] = normal(r, d, dtype=res, std=2.0) if case["residual"] else None
        s["next_weight"] = normal(d, dtype=f32, std=0.2, mean=1.0) if case["next"] else None
    # A program that keeps the states of its step calls apart has the room for the new ones in hand.
    if op.endswith("_step"):
        s["new_state"] = torch.empty_like(s["state"])
    return s


_SCALE, _EPS = 0.75, 1e-6


def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    import gated_deltanet_linear_chunk_gb300 as gdn
    case = s["case"]
    op = case["op"]
    if op == "conv":
        return gdn.gdn_short_conv(s["x"], s["weight"], s["cu"], bias=s["bias"], initial_state=s["state"],
                                  activation=s["act"], output_final_state=True)
    if op == "conv_step":
        out = gdn.gdn_short_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], activation=s["act"],
                                      new_state=s["new_state"])
        return out, s["new_state"]
    if op == "scan":
        return gdn.gdn_selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], D=s["D"], z=s["z"],
                                      dt_bias=s["dt_bias"], dt_softplus=True, initial_state=s["state"],
                                      output_final_state=True)
    if op == "scan_step":
        out = gdn.gdn_selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"],
                                          dt_bias=s["dt_bias"], dt_softplus=True, new_state=s["new_state"])
        return out, s["new_state"]
    return gdn.gdn_norm_gate_residual(s["y"], weight=s["weight"], gate=s["gate"], residual=s["residual"],
                                      next_weight=s["next_weight"], activation=case["act"],
                                      gate_first=case["first"], scale=_SCALE, eps=_EPS)


# ---- plain forms -----------------------------------------------------------------------------------------------


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _sequence_of(cu, tokens):
    """The sequence of each token."""
    return (torch.arange(tokens, device=cu.device)[:, None] >= cu[None, 1:]).sum(1)


def _conv_plain(s):
    x, cu, k = s["x"], s["cu"].long(), s["case"]["width"]
    tokens, c = x.shape
    seqs = cu.shape[0] - 1
    past = s["state"] if s["state"] is not None else x.new_zeros(seqs, k - 1, c)
    rows = torch.cat([x, past.reshape(seqs * (k - 1), c)])

    def place(seq, at):
        """The row of `rows` that holds position `at` of the packed tokens as sequence `seq` sees it."""
        before = at - cu[seq]
        return torch.where(before >= 0, at, tokens + seq * (k - 1) + (k - 1) + before)

    tap = torch.arange(k, device=x.device)
    seq = _sequence_of(cu, tokens)
    at = torch.arange(tokens, device=x.device)[:, None] - (k - 1) + tap
    y = (rows[place(seq[:, None].expand_as(at), at)].float() * s["weight"].t()[None]).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["act"]:
        y = y * _sigmoid(y)
    every = torch.arange(seqs, device=x.device)[:, None].expand(seqs, k - 1)
    return y.to(x.dtype), rows[place(every, cu[1:, None] - (k - 1) + tap[None, :k - 1])]


def _conv_step_plain(s):
    window = torch.cat([s["state"], s["x"][:, None]], dim=1)
    y = (window.float() * s["weight"].t()[None]).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["act"]:
        y = y * _sigmoid(y)
    return y.to(s["x"].dtype), window[:, 1:].contiguous()


def _scan_terms(s):
    """(decay, added) [rows, channels, states] of h_t = decay_t h_{t-1} + added_t."""
    v = s["dt"].float() + s["dt_bias"]
    step = torch.where(v > 20.0, v, torch.log1p(torch.exp(v)))
    decay = torch.exp(step[:, :, None] * s["A"][None])
    rows, g, n = s["B"].shape
    added = ((step * s["x"].float()).view(rows, g, -1, 1) * s["B"].float()[:, :, None, :]).view(rows, -1, n)
    return decay, added


def _scan_out(s, h):
    rows, g, n = s["C"].shape
    y = (h.view(rows, g, -1, n) * s["C"].float()[:, :, None, :]).sum(-1).view(rows, -1)
    if s["D"] is not None:
        y = y + s["D"] * s["x"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * _sigmoid(z))
    return y.to(s["x"].dtype)


def _scan_plain(s):
    a, h = _scan_terms(s)
    cu = s["cu"].long()
    seqs = cu.shape[0] - 1
    past = s["state"] if s["state"] is not None else a.new_zeros(seqs, *a.shape[1:])
    some = torch.nonzero(cu[1:] > cu[:-1])[:, 0]
    first = cu[some]
    h[first] += a[first] * past[some]
    a[first] = 0.0
    # The recurrence by doubling: after a round of distance d, (a, h) cover 2 d tokens.
    d = 1
    while d < s["longest"]:
        h[d:] += a[d:] * h[:-d]
        a[d:] = a[d:] * a[:-d]
        d *= 2
    final = past.clone()
    final[some] = h[cu[some + 1] - 1]
    return _scan_out(s, h), final


def _scan_step_plain(s):
    a, b = _scan_terms(s)
    h = a * s["state"] + b
    return _scan_out(s, h), h


def _norm_plain(s):
    case = s["case"]

    def normed(v, weight):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + _EPS) * weight

    m = s["y"].float()
    gate = None
    if s["gate"] is not None:
        gate = s["gate"].float()
        gate = _sigmoid(gate) * (gate if case["act"] == "silu" else 1.0)
    if gate is not None and case["first"]:
        m = m * gate
    if s["weight"] is not None:
        m = normed(m, s["weight"])
    if gate is not None and not case["first"]:
        m = m * gate
    m = m * _SCALE
    if s["residual"] is not None:
        m = m + s["residual"].float()
    return (m.to(_DTYPES[case["res"]]), None if s["next_weight"] is None else
            normed(m, s["next_weight"]).to(s["y"].dtype))


_PLAIN = {"conv": _conv_plain, "conv_step": _conv_step_plain, "scan": _scan_plain, "scan_step": _scan_step_plain,
          "norm": _norm_plain}


# ---- what a pass cannot do without -----------------------------------------------------------------------------


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("conv", "conv_step"):
        rows = case["tokens"] if op == "conv" else case["batch"]
        seqs = case["seqs"] if op == "conv" else case["batch"]
        c, k = case["channels"], case["width"]
        state = seqs * (k - 1) * c * e
        reads = state if op == "conv_step" or case["state"] else 0
        return {"bytes": 2 * rows * c * e + state + reads + 4 * c * (k + bool(case["bias"])),
                "flops": rows * c * (2 * k + (4 if case["silu"] else 0))}
    if op in ("scan", "scan_step"):
        rows = case["tokens"] if op == "scan" else case["batch"]
        seqs = case["seqs"] if op == "scan" else case["batch"]
        d, n, g = case["channels"], case["states"], case["groups"]
        state = seqs * d * n * 4
        reads = state if op == "scan_step" or case["state"] else 0
        each = rows * d * e * (3 + bool(case["gate"])) + 2 * rows * g * n * e
        # per state and token: the exponent's product and the exponential, the
        # term's product, the recurrence and the output sum
        return {"bytes": each + state + reads + 4 * d * (n + 1 + bool(case["skip"])), "flops": rows * d * (7 * n + 10)}
    r, d = case["rows"], case["dim"]
    f = 2 if case["res"] == "bf16" else 4
    return {"bytes": r * d * (e * (1 + bool(case["gate"]) + bool(case["next"])) + f * (1 + bool(case["residual"])))
            + 4 * d * (bool(case["weight"]) + bool(case["next"])),
            "flops": r * d * (4 * bool(case["weight"]) + 5 * bool(case["gate"]) + 2 + 4 * bool(case["next"]))}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------


def _wide(s):
    return {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}


def exact(case, seed):
    s = _wide(prepare(case, seed))
    op = case["op"]
    if op in ("conv", "conv_step"):
        k, rows = case["width"], s["x"].shape[0]
        cu = s["cu"].tolist() if op == "conv" else list(range(rows + 1))
        out, final = torch.empty_like(s["x"]), s["x"].new_empty(len(cu) - 1, k - 1, case["channels"])
        for i, (b, e) in enumerate(zip(cu[:-1], cu[1:])):
            past = s["state"][i] if s["state"] is not None else s["x"].new_zeros(k - 1, case["channels"])
            seen = torch.cat([past, s["x"][b:e]])
            y = sum(seen[j:j + e - b] * s["weight"][:, j] for j in range(k))
            y = y if s["bias"] is None else y + s["bias"]
            out[b:e] = torch.nn.functional.silu(y) if s["act"] else y
            final[i] = seen[e - b:]
        return out, final
    if op in ("scan", "scan_step"):
        rows, d = s["x"].shape
        cu = s["cu"].tolist() if op == "scan" else list(range(rows + 1))
        lens = [e - b for b, e in zip(cu[:-1], cu[1:])]
        order = sorted(range(len(lens)), key=lambda i: -lens[i])  # longest first: those still running are the first
        first = torch.tensor([cu[i] for i in order], device="cuda")
        h = s["state"][order] if s["state"] is not None else s["x"].new_zeros(len(lens), d, case["states"])
        step = torch.nn.functional.softplus(s["dt"] + s["dt_bias"], threshold=60.0)
        per = d // case["groups"]
        out = torch.empty_like(s["x"])
        for t in range(max(lens)):
            live = sum(n > t for n in lens) if len(lens) > 1 else 1
            at = first[:live] + t
            b, c = (s[v][at].repeat_interleave(per, dim=1) for v in ("B", "C"))
            q = step[at][:, :, None]
            h[:live] = torch.exp(q * s["A"]) * h[:live] + q * s["x"][at][:, :, None] * b
            out[at] = torch.einsum("rdn,rdn->rd", h[:live], c)
        if s["D"] is not None:
            out += s["D"] * s["x"]
        if s["z"] is not None:
            out *= torch.nn.functional.silu(s["z"])
        final = torch.empty_like(h)
        final[order] = h
        return out, final
    m = s["y"]
    gate = 1.0
    if s["gate"] is not None:
        gate = torch.nn.functional.silu(s["gate"]) if case["act"] == "silu" else torch.sigmoid(s["gate"])
    m = m * gate if case["first"] else m
    if s["weight"] is not None:
        m = m / torch.sqrt(torch.linalg.vector_norm(m, dim=1, keepdim=True) ** 2 / case["dim"] + _EPS) * s["weight"]
    m = m if case["first"] else m * gate
    m = _SCALE * m
    m = m if s["residual"] is None else s["residual"] + m
    if s["next_weight"] is None:
        return m, None
    return m, m / torch.sqrt(torch.linalg.vector_norm(m, dim=1, keepdim=True) ** 2 / case["dim"] + _EPS) * s["next_weight"]
