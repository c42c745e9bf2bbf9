"""Cases, plain forms and 64-bit values of the attention layers beside the fixed-state ones of a hybrid model.

The operators, with the entry points that a user calls for them:

* rope       gdn_qk_norm_rope: RMS norms of queries and keys for each head and
             their rotation by position (of one axis or several), in one pass
* append     gdn_paged_append: the same on the way of new keys and values into
             a paged cache, which may be 8-bit, over packed sequences
* attention  gdn_paged_attention: attention of one to eight new tokens of each
             sequence over its paged cache, with an output gate

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits (angles in 64), rounded once at the end; with ``own`` true it calls the
entry points.  ``exact`` evaluates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
_SIZES = {"bf16": 2, "f32": 4, "e4m3": 1}
_EPS, _THETA = 1e-6, 1e7

# Largest drawn sizes: bytes of the queries and keys, of the appended tensors
# and the cache beside them, of an attention's cache, and products of its scores.
_MOST_ROPE = 20480 * 40 * 128 * 2
_MOST_APPEND = 8192 * 40 * 256 * 2
_MOST_APPEND_CACHE = 1 << 29
_MOST_CACHE = 1 << 30
_MOST_PRODUCTS = 1 << 31


def listed():
    return [
        # A 4000-token prompt on its way to attention: queries with their output gates head by head in one
        # projection, a quarter of each head rotated.
        dict(name="rope_prompt", op="rope", dtype="bf16", tokens=4000, heads=24, kv_heads=4, dim=256, rotary=64,
             norm=True, axes=1, interleaved=False, gated=True),
        # Frames of a video: positions of three axes (time, height, width), whole heads rotated.
        dict(name="rope_video", op="rope", dtype="bf16", tokens=20480, heads=32, kv_heads=8, dim=128, rotary=128,
             norm=True, axes=3, interleaved=False, gated=False),
        # One token in fp32, heads of an odd width, neighbouring elements paired: the call's latency.
        dict(name="rope_token", op="rope", dtype="f32", tokens=1, heads=9, kv_heads=3, dim=74, rotary=38, norm=False,
             axes=1, interleaved=True, gated=False),
        # A full server's next tokens into the cache, with their queries.
        dict(name="append_batch", op="append", dtype="bf16", cache="bf16", tokens=64, seqs=64, longest=8192, page=16,
             heads=24, kv_heads=4, dim=256, rotary=64, norm=True, axes=1, interleaved=False, query=True, gated=True),
        # Prompts packed together, some empty or of one token, into an 8-bit cache.
        dict(name="append_prompts", op="append", dtype="bf16", cache="e4m3", tokens=8192, seqs=17, longest=8192,
             page=64, heads=24, kv_heads=4, dim=256, rotary=64, norm=True, axes=1, interleaved=False, query=True,
             gated=True),
        # Short prompts in fp32, an odd page size, keys that are rotated but not normed, no queries.
        dict(name="append_ragged", op="append", dtype="f32", cache="f32", tokens=999, seqs=41, longest=500, page=10,
             heads=6, kv_heads=2, dim=64, rotary=64, norm=False, axes=1, interleaved=True, query=False, gated=False),
        # A single user's next token after the 4000-token prompt: the call's latency.
        dict(name="attention_token", op="attention", dtype="bf16", cache="bf16", seqs=1, new=1, longest=4000,
             ragged=False, page=16, heads=24, kv_heads=4, dim=256, gate=True, lse=False),
        # A full server's next tokens, conversations of every length.
        dict(name="attention_batch", op="attention", dtype="bf16", cache="bf16", seqs=64, new=1, longest=8192,
             ragged=True, page=16, heads=24, kv_heads=4, dim=256, gate=True, lse=False),
        # One long document.
        dict(name="attention_long", op="attention", dtype="bf16", cache="bf16", seqs=1, new=1, longest=262144,
             ragged=False, page=64, heads=24, kv_heads=4, dim=256, gate=True, lse=False),
        # Eight drafted tokens of each sequence verified together.
        dict(name="attention_verify", op="attention", dtype="bf16", cache="bf16", seqs=32, new=8, longest=4000,
             ragged=True, page=16, heads=24, kv_heads=4, dim=256, gate=True, lse=False),
        # A fuller server on an 8-bit cache, narrower heads in larger groups.
        dict(name="attention_8bit", op="attention", dtype="bf16", cache="e4m3", seqs=128, new=1, longest=8192,
             ragged=True, page=32, heads=64, kv_heads=8, dim=128, gate=False, lse=False),
        # A few short sequences in fp32, an odd page size and an odd group, statistics returned.
        dict(name="attention_odd", op="attention", dtype="f32", cache="f32", seqs=5, new=3, longest=1001, ragged=True,
             page=10, heads=15, kv_heads=5, dim=64, gate=False, lse=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention"])
    coin = lambda: rng.random() < 0.5  # noqa: E731
    dtype = rng.choice(["bf16", "bf16", "f32"])
    cache = "f32" if dtype == "f32" else rng.choice(["bf16", "bf16", "e4m3"])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 6, 8, 16])
    if op == "rope":
        dim = rng.choice([64, 128, 256, 2 * _log(rng, 1, 256), 8 * _log(rng, 1, 64)])
        rotary = rng.choice([dim, dim, 2 * rng.randint(1, dim // 2), 0])
        most = _MOST_ROPE // ((heads + kv) * dim * _SIZES[dtype])
        return dict(op=op, dtype=dtype, tokens=max(1, min(_log(rng, 1, 70904), most)), heads=heads,
                    kv_heads=kv, dim=dim, rotary=rotary, norm=coin() or rotary == 0,
                    axes=rng.choice([1, 1, 2, 3]) if rotary else 1, interleaved=coin(), gated=coin())
    dim = rng.choice([64, 128, 256])
    page = rng.choice([16, 16, 32, 64, 128, _log(rng, 1, 256)])
    if op == "append":
        rotary = rng.choice([dim, dim // 4, 2 * rng.randint(1, dim // 2), 0])
        tokens = max(1, min(_log(rng, 1, 20000), _MOST_APPEND // ((heads + 4 * kv) * dim * _SIZES[dtype])))
        seqs = rng.choice([1, min(tokens, 512), _log(rng, 1, 200)])
        tokens = seqs if seqs == 512 else tokens
        longest = max(1, min(_log(rng, 64, 8192), _MOST_APPEND_CACHE // (2 * seqs * kv * dim * _SIZES[cache])))
        return dict(op=op, dtype=dtype, cache=cache, tokens=tokens, seqs=seqs, longest=longest, page=page, heads=heads,
                    kv_heads=kv, dim=dim, rotary=rotary, norm=coin(),
                    axes=rng.choice([1, 1, 1, 3]) if rotary else 1, interleaved=coin(), query=coin(), gated=coin())
    seqs, new = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 3, 4, 8])
    longest = max(1, min(_log(rng, 1, 131072), _MOST_CACHE // (2 * seqs * kv * dim * _SIZES[cache]),
                         _MOST_PRODUCTS // (seqs * heads * new * dim)))
    return dict(op=op, dtype=dtype, cache=cache, seqs=seqs, new=new, longest=longest, ragged=coin(), page=page,
                heads=heads, kv_heads=kv, dim=dim, gate=coin(), lse=coin())


def _lengths(case):
    """How many tokens of each sequence are new, and how many the cache then holds of each: spread over the
    logarithm, empty ones and single tokens among them."""
    seqs, longest = case["seqs"], case["longest"]
    if case["op"] == "attention":
        rng = random.Random(longest * 1000003 + seqs)
        if not case["ragged"]:
            return [case["new"]] * seqs, [longest] * seqs
        lens = [0 if rng.random() < 0.03 else _log(rng, max(1, longest // 64), longest) for _ in range(seqs)]
        lens[rng.randrange(seqs)] = longest
        return [case["new"]] * seqs, lens
    tokens = case["tokens"]
    rng = random.Random(tokens * 1000003 + seqs)
    if seqs == tokens:
        new = [1] * seqs
    else:
        shares = [0.0 if rng.random() < 0.1 else math.exp(rng.uniform(0.0, 4.0)) for _ in range(seqs)]
        shares[rng.randrange(seqs)] += 1.0
        total, new, used, seen = sum(shares), [], 0, 0.0
        for s in shares:
            seen += s
            end = int(round(tokens * seen / total))
            new.append(end - used)
            used = end
    # Prompts start a conversation or go on with one.
    return new, [n + (rng.randint(0, longest - n) if n < longest and (n == 1 or rng.random() < 0.5) else 0)
                 for n in new]


def _axes(case):
    """The axis of each pair's angle: those of a head in turn, as height and width alternate within time's."""
    return [i % case["axes"] for i in range(case["rotary"] // 2)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, f32 = _DTYPES[case["dtype"]], torch.float32

    def normal(*shape, dtype=dt, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    op, dim, kv = case["op"], case["dim"], case["kv_heads"]
    s = {"case": case, "scale": dim ** -0.5}

    def queries(*lead, gated):
        """Queries and the gates of their outputs, head by head in one projection, or queries alone."""
        both = normal(*lead, case["heads"], dim * (2 if gated else 1))
        return both[..., :dim], (both[..., dim:] if gated else None)

    if op != "attention":
        tokens, rotary = case["tokens"], case["rotary"]
        s["q"], _ = queries(tokens, gated=case["gated"])
        # Keys and values are columns of one projection.
        k, s["v"] = normal(tokens, 2 * kv * dim).view(tokens, 2, kv, dim).unbind(1)
        s["k"] = k
        s["q_weight"] = normal(dim, dtype=f32, std=0.2, mean=1.0) if case["norm"] else None
        s["k_weight"] = normal(dim, dtype=f32, std=0.2, mean=1.0) if case["norm"] else None
        s["inv_freq"] = (_THETA ** (-torch.arange(0, rotary, 2, device="cuda", dtype=torch.float64) / rotary)).float() \
            if rotary else None
        s["axes"] = _axes(case) if case["axes"] > 1 else None
        if op == "rope" or case["axes"] > 1:
            far = 262144 if case["axes"] == 1 else 4096
            shape = (tokens,) if case["axes"] == 1 else (case["axes"], tokens)
            s["positions"] = torch.randint(0, far, shape, generator=gen, device="cuda").to(torch.int32)
        else:
            s["positions"] = None
    if op != "rope":
        new, lens = _lengths(case)
        page, ct = case["page"], _DTYPES[case["cache"]]
        used = [-(-n // page) for n in lens]
        width, pages = max(max(used), 1) + 1, sum(used) + 3
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        ends = torch.tensor(used, device="cuda").cumsum(0)
        at = torch.arange(width, device="cuda")[None] + (ends - torch.tensor(used, device="cuda"))[:, None]
        within = torch.arange(width, device="cuda")[None] < torch.tensor(used, device="cuda")[:, None]
        s["page_table"] = torch.where(within, order[at.clamp(max=pages - 1)], -1).to(torch.int32)
        s["seq_lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        s["longest"] = max(lens)
        eight = case["cache"] == "e4m3"
        # Head by head within a page.
        s["k_cache"] = normal(pages, kv, page, dim, dtype=ct, std=32.0 if eight else 1.0).transpose(1, 2)
        s["v_cache"] = normal(pages, kv, page, dim, dtype=ct, std=32.0 if eight else 1.0).transpose(1, 2)
        s["k_scale"] = (torch.rand(kv, generator=gen, device="cuda") + 0.5) / 32 if eight else None
        s["v_scale"] = (torch.rand(kv, generator=gen, device="cuda") + 0.5) / 32 if eight else None
        if op == "append":
            s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
        else:
            s["q"], s["gate"] = queries(case["seqs"], case["new"], gated=case["gate"])
            s["q"] = s["q"].contiguous()  # as gdn_paged_append returns them
    return s


def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    import gated_deltanet_linear_chunk_gb300 as gdn
    case = s["case"]
    if case["op"] == "rope":
        return gdn.gdn_qk_norm_rope(s["q"], s["k"], positions=s["positions"] if case["rotary"] else None,
                                    inv_freq=s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=_EPS,
                                    axes=s["axes"], interleaved=case["interleaved"])
    if case["op"] == "append":
        q = gdn.gdn_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"],
                                 cu_seqlens=s["cu"], q=s["q"] if case["query"] else None, positions=s["positions"],
                                 inv_freq=s["inv_freq"], q_weight=s["q_weight"] if case["query"] else None,
                                 k_weight=s["k_weight"], eps=_EPS, axes=s["axes"], interleaved=case["interleaved"],
                                 k_scale=s["k_scale"], v_scale=s["v_scale"])
        return q, s["k_cache"], s["v_cache"]
    return gdn.gdn_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"],
                                   scale=s["scale"], gate=s["gate"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                   return_lse=case["lse"])


# ---- plain forms -----------------------------------------------------------------------------------------------


def _norm_rotate(s, x, weight, positions):
    """x [T, H, D] normed and rotated, in 32 bits."""
    case = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * weight
    if not case["rotary"]:
        return x
    half = case["rotary"] // 2
    where = positions[s["axes"]] if s["axes"] else positions[None].expand(half, -1)
    angle = where.t().double() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _rope_plain(s):
    dt = s["q"].dtype
    return (_norm_rotate(s, s["q"], s["q_weight"], s["positions"]).to(dt),
            _norm_rotate(s, s["k"], s["k_weight"], s["positions"]).to(dt))


def _places(s):
    """For each packed token its index in its sequence, the page and the place in the page."""
    cu, page = s["cu"].long(), s["case"]["page"]
    token = torch.arange(s["k"].shape[0], device=cu.device)
    seq = (token[:, None] >= cu[None, 1:]).sum(1)
    index = s["seq_lens"].long()[seq] - cu[seq + 1] + token
    return index, s["page_table"].long()[seq, index // page], index % page


def _stored(x, scale, dtype):
    if scale is None:
        return x.to(dtype)
    return (x / scale[:, None]).clamp(-448.0, 448.0).to(dtype)


def _append_plain(s):
    case = s["case"]
    index, page, slot = _places(s)
    where = index if s["positions"] is None else s["positions"]
    for cache, x, scale in ((s["k_cache"], _norm_rotate(s, s["k"], s["k_weight"], where), s["k_scale"]),
                            (s["v_cache"], s["v"].float(), s["v_scale"])):
        x = _stored(x, scale, cache.dtype)
        if scale is None:
            cache[page, slot] = x
        else:  # whole bytes are moved
            cache.view(torch.uint8)[page, slot] = x.view(torch.uint8)
    q = _norm_rotate(s, s["q"], s["q_weight"], where).to(s["q"].dtype) if case["query"] else None
    return q, s["k_cache"], s["v_cache"]


def _pages(cache, at):
    """cache[at]; of an 8-bit cache whole bytes are moved."""
    return cache[at] if cache.element_size() > 1 else cache.view(torch.uint8)[at].view(cache.dtype)


def _gathered(s, cache, scale):
    """The first tokens of every sequence, [N, kv_heads, longest, D] in 32 bits."""
    page = s["case"]["page"]
    wide = -(-max(s["longest"], 1) // page)
    table = s["page_table"][:, :wide].long().clamp(min=0)
    x = _pages(cache, table).flatten(1, 2)
    x = x[:, :max(s["longest"], 1)].transpose(1, 2).float()
    return x if scale is None else x * scale[:, None, None]


def _attention_plain(s):
    case, q = s["case"], s["q"]
    n, new, heads, dim = q.shape
    kv = case["kv_heads"]
    k = _gathered(s, s["k_cache"], s["k_scale"])
    span = k.shape[2]
    rows = q.float().view(n, new, kv, heads // kv, dim).permute(0, 2, 1, 3, 4).reshape(n, kv, -1, dim)
    scores = (rows @ k.transpose(2, 3) * s["scale"]).view(n, kv, new, heads // kv, span)
    del k
    sees = s["seq_lens"].long()[:, None] - new + 1 + torch.arange(new, device=q.device)
    seen = torch.arange(span, device=q.device) < sees[..., None]
    scores = torch.where(seen[:, None, :, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    v = _gathered(s, s["v_cache"], s["v_scale"])
    v = torch.where((torch.arange(span, device=q.device) < s["seq_lens"][:, None])[:, None, :, None], v, 0.0)
    out = (p.view(n, kv, -1, span) @ v).view(n, kv, new, heads // kv, dim)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 2, 1, 3, 4).reshape(n, new, heads, dim)
    if s["gate"] is not None:
        out = out / (1.0 + torch.exp(-s["gate"].float()))
    out = out.to(q.dtype)
    if not case["lse"]:
        return out
    return out, (torch.log(total) + top)[..., 0].permute(0, 2, 1, 3).reshape(n, new, heads)


_PLAIN = {"rope": _rope_plain, "append": _append_plain, "attention": _attention_plain}


# ---- what a pass cannot do without -----------------------------------------------------------------------------


def work(case):
    e, dim, kv = _SIZES[case["dtype"]], case["dim"], case["kv_heads"]
    if case["op"] == "rope":
        rows, rotary = case["tokens"] * (case["heads"] + kv), case["rotary"]
        return {"bytes": 2 * rows * dim * e + 4 * (2 * dim * case["norm"] + rotary // 2
                                                   + (case["tokens"] * case["axes"] if rotary else 0)),
                "flops": rows * (4 * dim * case["norm"] + 3 * rotary)}
    new, lens = _lengths(case)
    c = _SIZES[case["cache"]]
    if case["op"] == "append":
        tokens, rotary = case["tokens"], case["rotary"]
        rows = tokens * (kv + case["heads"] * case["query"])
        return {"bytes": tokens * dim * (2 * kv * (e + c) + 2 * case["heads"] * case["query"] * e)
                + 4 * (tokens + 2 * case["seqs"] + 1 + dim * case["norm"] * (1 + case["query"]) + rotary // 2),
                "flops": rows * (4 * dim * case["norm"] + 3 * rotary) + 2 * tokens * kv * dim * (case["cache"] == "e4m3")}
    rows = case["seqs"] * case["new"] * case["heads"]
    seen = sum(max(0, n - case["new"] + 1 + t) for n in lens for t in range(case["new"])) * case["heads"]
    return {"bytes": 2 * sum(lens) * kv * dim * c + rows * (dim * e * (2 + case["gate"]) + 4 * case["lse"])
            + 4 * (case["seqs"] + sum(-(-n // case["page"]) for n in lens)),
            "flops": seen * (4 * dim + 4) + rows * dim * (1 + 4 * case["gate"])}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------


def _turned(s, x, weight, positions):
    """The definition head by head: pairs of elements as complex numbers, times e^(i angle)."""
    case = s["case"]
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["dim"] + _EPS) * weight.double()
    half = case["rotary"] // 2
    if half == 0:
        return y
    axis = torch.tensor(_axes(case), device=x.device)
    per = positions.reshape(case["axes"], -1).double()
    angle = per.index_select(0, axis).T * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    first = torch.arange(half, device=x.device) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y = y.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return (_turned(s, s["q"], s["q_weight"], s["positions"]), _turned(s, s["k"], s["k_weight"], s["positions"]))
    page, table = case["page"], s["page_table"].tolist()
    lens = s["seq_lens"].tolist()
    if case["op"] == "append":
        cu = s["cu"].tolist()
        index, at = [], []
        for i, (b, e) in enumerate(zip(cu[:-1], cu[1:])):
            for j in range(lens[i] - (e - b), lens[i]):
                index.append(j)
                at.append(table[i][j // page] * page + j % page)
        index = torch.tensor(index, device="cuda", dtype=torch.int64)
        at = torch.tensor(at, device="cuda", dtype=torch.int64)
        where = index if s["positions"] is None else s["positions"]
        q = _turned(s, s["q"], s["q_weight"], where) if case["query"] else None
        got = [q]
        for cache, x, scale in ((s["k_cache"], _turned(s, s["k"], s["k_weight"], where), s["k_scale"]),
                                (s["v_cache"], s["v"].double(), s["v_scale"])):
            if scale is not None:
                x = (x / scale.double()[None, :, None]).clamp(-448.0, 448.0)
            whole = cache.to(torch.float64).reshape(-1, case["kv_heads"], case["dim"])
            whole[at] = x
            got.append(whole.view(cache.shape))
        return tuple(got)
    n, new, heads, dim = s["q"].shape
    kv = case["kv_heads"]
    out = torch.zeros(n, new, heads, dim, device="cuda", dtype=torch.float64)
    lse = torch.full((n, new, heads), -math.inf, device="cuda", dtype=torch.float64)
    q = s["q"].double().view(n, new, kv, heads // kv, dim)
    for i, length in enumerate(lens):
        if length == 0:
            continue
        pages = torch.tensor(table[i][:-(-length // page)], device="cuda")
        held = []
        for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
            x = _pages(cache, pages).double().flatten(0, 1)[:length]
            held.append(x if scale is None else x * scale.double()[:, None])
        for t in range(new):
            sees = length - new + 1 + t
            if sees <= 0:
                continue
            scores = torch.einsum("hgd,shd->hgs", q[i, t], held[0][:sees]) * s["scale"]
            out[i, t] = torch.einsum("hgs,shd->hgd", torch.softmax(scores, -1), held[1][:sees]).reshape(heads, dim)
            lse[i, t] = torch.logsumexp(scores, -1).reshape(heads)
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].double())
    return (out, lse) if case["lse"] else out
