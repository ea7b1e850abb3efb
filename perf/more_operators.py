"""Cases for the mixer half of a block, between the norm and the int4 mixture-of-experts layer: the
int8 projection, rotary positions, linear attention with a decay for each head, and the norm after a
block with its gate, residual scale and the next block's norm.

`run` computes an operator in elementary torch operations (`own` false) or through the binding
(`own` true); `exact` evaluates the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
QMAX = {"int8": 127.0, "e4m3": 448.0}
CHUNK = 64  # tokens of a chunk in the plain form of linear attention


def _int8(name, T, N, K, dtype="bf16", bias=False, pad=0):
    return {"name": name, "op": "int8", "T": T, "N": N, "K": K, "dtype": dtype, "bias": bias, "pad": pad}


def _rope(name, T, q_heads, k_heads, D, rot, dtype="bf16", interleaved=False, scaling="none", factor=1.0, requests=1,
          context=32768, base=10000.0):
    return {"name": name, "op": "rope", "T": T, "q_heads": q_heads, "k_heads": k_heads, "D": D, "rot": rot, "dtype": dtype,
            "interleaved": interleaved, "scaling": scaling, "factor": factor, "requests": requests, "context": context,
            "base": base}


def _linear(name, T, seqs, k_heads, v_heads, dk, dv, per_token=True, step=False, fresh=0.5, pad=0):
    return {"name": name, "op": "linear", "T": T, "seqs": seqs, "k_heads": k_heads, "v_heads": v_heads, "dk": dk, "dv": dv,
            "per_token": per_token, "step": step, "fresh": fresh, "pad": pad}


def _gnorm(name, T, H, group=0, dtype="bf16", weight="bf16", gate="none", residual=False, after=True, channel=False,
           scale=1.0, following=False, out8="none", out8_group=0, offset=0.0, pad=0):
    return {"name": name, "op": "gnorm", "T": T, "H": H, "group": group, "dtype": dtype, "weight": weight, "gate": gate,
            "residual": residual, "after": after, "channel": channel, "scale": scale, "following": following, "out8": out8,
            "out8_group": out8_group, "offset": offset, "pad": pad}


def listed():
    return [
        # one decoded token into queries, keys, values and gates together
        _int8("int8 token", 1, 12288, 2048),
        # an attention's output projection of some requests' prompts, to f16, rows out of a wider buffer
        _int8("int8 prompts", 500, 2000, 4096, dtype="f16", bias=True, pad=64),
        # a long prefill chunk into queries, keys, values and gates together
        _int8("int8 long", 4096, 12288, 2048),
        # one decoded token, a quarter of each head turned, scaled to four times the trained context
        _rope("rope token", 1, 16, 2, 256, 64, scaling="yarn", factor=4.0, base=1e7),
        # a long prompt's chunk, whole heads turned in neighbouring pairs
        _rope("rope long", 16384, 32, 8, 128, 128, interleaved=True, requests=3),
        # one decoded token of one request
        _linear("linear token", 1, 1, 16, 32, 128, 128, step=True),
        # one decoding step of 48 requests
        _linear("linear batch", 48, 48, 16, 32, 128, 128, step=True),
        # prompts of several requests, some of them continued from a kept state, odd head sizes and a fixed decay a head
        _linear("linear prompts", 1777, 7, 6, 12, 96, 80, per_token=False, pad=8),
        # a long prompt beside a few short ones
        _linear("linear long", 16384, 4, 16, 32, 128, 128),
        # one decoded token's heads, normed, gated and put in 8 bits for the output projection
        _gnorm("gnorm token", 1, 4096, group=128, gate="silu", out8="int8"),
        # the same heads of a prompt, fp16 with an fp32 weight, rows of a wider buffer
        _gnorm("gnorm heads", 1500, 4096, group=128, dtype="f16", weight="f32", gate="sigmoid", out8="int8", pad=24),
        # the end of a block and the start of the next for a long prompt, with 8-bit rows for the next projection
        _gnorm("gnorm block", 16384, 2048, residual=True, scale=0.5, channel=True, following=True, out8="int8", offset=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["int8", "rope", "linear", "linear", "gnorm"])
    if op == "int8":
        N, K = _log_int(rng, 64, 12288), 64 * _log_int(rng, 4, 128)
        if rng.random() < 0.6:
            N = max(64, N // 64 * 64)
        T = _log_int(rng, 1, min(8192, 4096 * 12288 * 2048 // (N * K)))
        c = _int8("", T, N, K, rng.choice(["bf16", "bf16", "f16", "f32"]), rng.random() < 0.3, rng.choice([0, 0, 64]))
    elif op == "rope":
        D = 8 * rng.randint(4, 32)
        rot = D if rng.random() < 0.5 else 2 * rng.randint(4, D // 2)
        k_heads = rng.choice([1, 2, 4, 8])
        q_heads = k_heads * rng.randint(1, 8)
        T = _log_int(rng, 1, min(65536, 16384 * 40 * 128 // ((q_heads + k_heads) * D)))
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if dtype == "f32":
            T = max(1, T // 2)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        c = _rope("", T, q_heads, k_heads, D, rot, dtype, rng.random() < 0.5, scaling,
                  1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.5]), _log_int(rng, 1, min(T, 64)),
                  rng.choice([4096, 32768, 1 << 20]), rng.choice([1e4, 5e5, 1e7]))
    elif op == "linear":
        k_heads = rng.choice([1, 2, 4, 8, 16])
        v_heads = k_heads * rng.choice([1, 2, 4])
        dk, dv = 8 * rng.randint(4, 32), 8 * rng.randint(4, 32)
        if rng.random() < 0.5:
            dk, dv = rng.choice([64, 128]), rng.choice([64, 128])
        step = rng.random() < 0.4
        if step:
            T = seqs = _log_int(rng, 1, max(1, min(256, 48 * 32 * 128 * 128 // (v_heads * dk * dv))))
        else:
            T = _log_int(rng, 2, min(32768, 16384 * 32 * 128 // (v_heads * max(dk, dv))))
            seqs = _log_int(rng, 1, min(T, 64))
        c = _linear("", T, seqs, k_heads, v_heads, dk, dv, rng.random() < 0.7, step, rng.choice([0.0, 0.5, 1.0]),
                    rng.choice([0, 0, 8]))
    else:
        H = _log_int(rng, 128, 8192)
        group = rng.choice([0, 0, 64, 128])
        out8 = rng.choice(["none", "none", "int8", "e4m3"])
        out8_group = rng.choice([0, 0, 128]) if out8 != "none" else 0
        if group or out8_group or rng.random() < 0.7:
            H = max(128, H // 128 * 128)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        T = _log_int(rng, 1, (8192 if dtype == "f32" else 16384) * 2048 // H)
        after = rng.random() < 0.8
        c = _gnorm("", T, H, group if after else 0, dtype, rng.choice([dtype, "f32"]),
                   rng.choice(["none", "silu", "sigmoid", "row"]), rng.random() < 0.6, after, rng.random() < 0.4,
                   rng.choice([1.0, 0.22]), rng.random() < 0.6, out8, out8_group, rng.choice([0.0, 1.0]), rng.choice([0, 0, 8, 3]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rows(t, pad, dtype):
    """t in rows of its width and `pad` values more."""
    return torch.cat([t, t[:, :pad]], 1).to(dtype)[:, :t.shape[1]] if pad else t.to(dtype)


def _new(T, width, pad, dtype):
    return torch.empty((T, width + pad), dtype=dtype, device="cuda")[:, :width]


def _prepare_int8(c, g):
    T, N, K = c["T"], c["N"], c["K"]
    # rows as a norm leaves them: the largest value of each at 127, most far below it
    x = _normal(g, T, K)
    x = x * (127 / x.abs().amax(1, keepdim=True))
    w = _normal(g, N, K)
    w = w * (127 / w.abs().amax(1, keepdim=True))
    s = {"c": c, "x": _rows(x.round(), c["pad"], torch.int8), "w": w.round().to(torch.int8)}
    s["x_scales"] = torch.rand(T, generator=g, device="cuda") * 0.03 + 0.01
    s["w_scales"] = (torch.rand(N, generator=g, device="cuda") * 0.5 + 0.75) * 0.03 / math.sqrt(K)
    s["bias"] = _normal(g, N) * 0.1 if c["bias"] else None
    if own:
        s["y"] = _new(T, N, 0, TYPES[c["dtype"]])
        from int4_grouped_gemm_router_amd import binding as B
        s["ws"] = B.project_int8_workspace(N, K, T)
    return s


def _runs(T, n, g):
    """Lengths of n runs of one value at least that make up T, a few of them much longer than the others, and their ends."""
    share = torch.exp(_normal(g, n) * 1.2)
    ends = (share.cumsum(0) / share.sum() * (T - n)).round().long() + torch.arange(1, n + 1, device="cuda")
    ends[-1] = T
    return torch.cat([ends.new_zeros(1), ends])


def _prepare_rope(c, g):
    T, Hq, Hk, D = c["T"], c["q_heads"], c["k_heads"], c["D"]
    # queries, keys and values of one projection, a row a token
    qkv = _normal(g, T, (Hq + 2 * Hk) * D).to(TYPES[c["dtype"]])
    s = {"c": c, "q": qkv[:, :Hq * D].view(T, Hq, D), "k": qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)}
    cu = _runs(T, c["requests"], g)
    begin = torch.randint(0, c["context"], (c["requests"],), generator=g, device="cuda")
    of = torch.searchsorted(cu[1:], torch.arange(T, device="cuda"), right=True)
    s["positions"] = (torch.arange(T, device="cuda") - cu[:-1][of] + begin[of]).to(torch.int32)
    s["inv_freq"], s["magnitude"] = _frequencies(c)
    if own:
        from int4_grouped_gemm_router_amd import binding as B
        s["plan"] = B.rope(D, c["rot"], dtype=TYPES[c["dtype"]], interleaved=c["interleaved"], base=c["base"],
                           scaling={"none": B.ROPE_PLAIN, "linear": B.ROPE_LINEAR, "ntk": B.ROPE_NTK,
                                    "yarn": B.ROPE_YARN}[c["scaling"]],
                           factor=c["factor"], context=c["context"])
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    return s


def _prepare_linear(c, g):
    T, n, Hk, Hv, dk, dv, pad = (c[k] for k in ("T", "seqs", "k_heads", "v_heads", "dk", "dv", "pad"))
    unit = lambda t: t / t.square().sum(2, keepdim=True).sqrt()  # noqa: E731
    bf16 = torch.bfloat16
    s = {"c": c, "q": _rows(unit(_normal(g, T, Hk, dk)).view(T, -1), pad, bf16).view(T, Hk, dk),
         "k": _rows(unit(_normal(g, T, Hk, dk)).view(T, -1), pad, bf16).view(T, Hk, dk),
         "v": _rows(_normal(g, T, Hv * dv), pad, bf16).view(T, Hv, dv)}
    # heads that remember from a few tokens to some thousands
    per_head = -torch.exp(-torch.linspace(1.0, 8.0, Hv, device="cuda"))
    s["decay"] = per_head * torch.exp(_normal(g, T, Hv) * 0.5) if c["per_token"] else per_head
    s["cu"] = torch.arange(T + 1, device="cuda") if c["step"] else _runs(T, n, g)
    slots = n + 3
    s["pool"] = _normal(g, slots, Hv, dk, dv) * 0.3
    s["slots"] = torch.randperm(slots, generator=g, device="cuda")[:n]
    if not c["step"]:
        s["slots"] = torch.where(torch.rand(n, generator=g, device="cuda") < c["fresh"], -1, s["slots"])
    s["cu"], s["slots"] = s["cu"].to(torch.int32), s["slots"].to(torch.int32)
    s["scale"] = 1.0
    if own:
        from int4_grouped_gemm_router_amd import binding as B
        s["plan"] = B.linear_attention(Hk, Hv, dk, dv, scale=s["scale"])
        s["o"] = torch.empty((T, Hv, dv), dtype=bf16, device="cuda")
        s["state"] = torch.empty((n, Hv, dk, dv), device="cuda")
        s["ws"] = None if c["step"] else B.linear_attention_workspace(s["plan"], n, T)
    return s


def _prepare_gnorm(c, g):
    dt, T, H, pad = TYPES[c["dtype"]], c["T"], c["H"], c["pad"]
    wt = TYPES[c["weight"]]
    G = c["group"] or H
    s = {"c": c, "x": _rows(_normal(g, T, H) * torch.exp(_normal(g, T, 1) * 0.5), pad, dt)}
    weight = lambda n: (torch.rand(n, generator=g, device="cuda") * 0.5 + 0.75 - c["offset"]).to(wt)  # noqa: E731
    s["weight"] = weight(G) if c["after"] else None
    s["gate"] = None
    if c["gate"] != "none":
        s["gate"] = _normal(g, T, 1).to(dt) if c["gate"] == "row" else _rows(_normal(g, T, H), pad, dt)
    s["channel"] = (torch.rand(H, generator=g, device="cuda") + 0.5).to(wt) if c["channel"] else None
    # a residual stream, a few channels of it much larger than the rest
    s["residual"] = None
    if c["residual"]:
        channel = torch.ones(H, device="cuda")
        channel[torch.randint(0, H, (max(1, H // 256),), generator=g, device="cuda")] = 20.0
        s["residual"] = _rows(_normal(g, T, H) * channel, pad, dt)
    s["next"] = weight(H) if c["following"] else None
    if own:
        from int4_grouped_gemm_router_amd import binding as B
        kind = {"none": B.GATE_NONE, "silu": B.GATE_SILU, "sigmoid": B.GATE_SIGMOID, "row": B.GATE_SIGMOID}[c["gate"]]
        s["plan"] = B.gated_norm(H, dtype=dt, weight_dtype=wt, normalize=c["after"], group=c["group"], eps=EPS,
                                 weight_offset=c["offset"], gate=kind, gate_per_row=c["gate"] == "row", scale=c["scale"],
                                 next_norm=c["following"], next_eps=EPS, next_offset=c["offset"],
                                 out8={"none": B.OUT8_NONE, "int8": B.OUT8_INT8, "e4m3": B.OUT8_E4M3}[c["out8"]],
                                 out8_group=c["out8_group"])
        s["h"] = _new(T, H, pad, dt)
        s["y"] = _new(T, H, pad, dt) if c["following"] else None
        s["q"] = s["q_scales"] = None
        if c["out8"] != "none":
            s["q"] = torch.empty((T, H), dtype=torch.int8 if c["out8"] == "int8" else torch.float8_e4m3fn, device="cuda")
            s["q_scales"] = torch.empty((T, H // c["out8_group"] if c["out8_group"] else 1), device="cuda")
            s["values"] = torch.empty((T, H), dtype=dt, device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"int8": _prepare_int8, "rope": _prepare_rope, "linear": _prepare_linear, "gnorm": _prepare_gnorm}[case["op"]](case, g)


# ------------------------------------------------------------------ the plain forms

def _plain_int8(s):
    y = s["x"].float() @ s["w"].float().t()  # whole numbers, exact in 32 bits up to 2^24
    y = y * s["x_scales"][:, None] * s["w_scales"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(TYPES[s["c"]["dtype"]])}


def _frequencies(c):
    """Radians a position turns each pair by, in 64 bits, and the factor on cosine and sine."""
    rot, f = c["rot"], c["factor"]
    power = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot
    base = c["base"] * f ** (rot / (rot - 2)) if c["scaling"] == "ntk" else c["base"]
    inv = base ** -power
    if c["scaling"] == "linear":
        return inv / f, 1.0
    if c["scaling"] != "yarn":
        return inv, 1.0
    turns = c["context"] * inv / (2 * math.pi)  # of a pair over the trained context: below 1 stretched, above 32 kept
    kept = ((turns - 1) / 31).clamp(0, 1)
    return inv * kept + inv / f * (1 - kept), 0.1 * math.log(f) + 1


def _plain_rope(s):
    c, out = s["c"], {}
    rot = c["rot"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    for name in ("q", "k"):
        x = s[name]
        t = x[..., :rot].float()
        a, b = (t[..., ::2], t[..., 1::2]) if c["interleaved"] else (t[..., :rot // 2], t[..., rot // 2:])
        turned = [a * cos - b * sin, a * sin + b * cos]
        t = torch.stack(turned, -1).flatten(-2) if c["interleaved"] else torch.cat(turned, -1)
        out[name] = torch.cat([t.to(x.dtype), x[..., rot:]], -1)
    return out


def _first_states(s):
    c = s["c"]
    kept = (s["slots"] >= 0).float()
    return s["pool"][s["slots"].clamp(min=0).long()] * kept[:, None, None, None]


def _plain_linear(s):
    c = s["c"]
    T, n, Hv, dk, dv = (c[k] for k in ("T", "seqs", "v_heads", "dk", "dv"))
    each = Hv // c["k_heads"]
    q, k = (s[x].float().repeat_interleave(each, 1) for x in "qk")
    v, S = s["v"].float(), _first_states(s)
    g = s["decay"].expand(T, Hv)
    if c["step"]:
        S = S * torch.exp(g)[:, :, None, None] + k[..., None] * v[:, :, None, :]
        return {"o": (s["scale"] * (q[..., None] * S).sum(2)).to(torch.bfloat16), "state": S}
    # each sequence in chunks of its own: the token at each place of each chunk, and whether there is one
    cu = s["cu"].long()
    chunks = (cu[1:] - cu[:-1] + CHUNK - 1) // CHUNK
    ends = chunks.cumsum(0)
    m = T // CHUNK + n
    j = torch.arange(m, device="cuda")
    of = torch.searchsorted(ends, j, right=True).clamp(max=n - 1)
    at = cu[of] + (j - (ends - chunks)[of]) * CHUNK
    rows = at[:, None] + torch.arange(CHUNK, device="cuda")
    there = (rows < cu[of + 1][:, None]) & (j < ends[-1])[:, None]
    rows = torch.where(there, rows, 0)
    held = there.float()[:, :, None]
    q, k, v = ((t[rows] * held[..., None]).permute(0, 2, 1, 3) for t in (q, k, v))  # [m, Hv, CHUNK, d]
    G = (g.double()[rows] * held).cumsum(1).permute(0, 2, 1)  # [m, Hv, CHUNK]
    total = G[:, :, -1]
    # what each chunk adds to the state, and what of it is left at the start of each later one of its sequence
    added = (k * torch.exp(total[..., None] - G).float()[..., None]).transpose(2, 3).contiguous() @ v
    first = (j == (ends - chunks)[of]).double()[:, None] * (j < ends[-1])[:, None]
    before = total.cumsum(0) - total
    left = (before[:, None] - before[None, :] - total[None, :])  # [to, from, Hv]
    same = (of[:, None] == of[None, :]) & (j[:, None] > j[None, :])
    left = torch.where(same[..., None], torch.exp(left.clamp(max=0)), 0).float()
    start = torch.zeros_like(before).index_add(0, of, before * first)[of]  # the sum before the sequence's first chunk
    kept = torch.exp((before - start).clamp(max=0)).float()
    S = kept[..., None, None] * S[of] + (left.permute(2, 0, 1).contiguous() @ added.view(m, Hv, -1).transpose(0, 1).contiguous()
                                        ).transpose(0, 1).view(m, Hv, dk, dv)
    near = G[..., :, None] - G[..., None, :]
    causal = torch.ones((CHUNK, CHUNK), device="cuda").tril()
    near = torch.exp(near.clamp(max=0)).float() * causal
    o = (q * torch.exp(G).float()[..., None]) @ S + ((q @ k.transpose(2, 3).contiguous()) * near) @ v
    S = S * torch.exp(total).float()[..., None, None] + added  # after each chunk
    out = torch.zeros((T, Hv, dv), dtype=torch.bfloat16, device="cuda")
    out[rows[there]] = (s["scale"] * o).permute(0, 2, 1, 3)[there].to(torch.bfloat16)
    return {"o": out, "state": S[ends - 1]}


def _plain_gnorm(s):
    c, out = s["c"], {}
    T, H, G = c["T"], c["H"], c["group"] or c["H"]
    dt = s["x"].dtype
    m = s["x"].float()
    if c["after"]:
        f = m.view(T, -1, G)
        m = (f * torch.rsqrt((f * f).mean(2, keepdim=True) + EPS) * (s["weight"].float() + c["offset"])).view(T, H)
    if c["gate"] != "none":
        z = s["gate"].float()
        m = m * (1 / (1 + torch.exp(-z))) * (z if c["gate"] == "silu" else 1.0)
    if c["channel"]:
        m = m * s["channel"].float()
    v = m * c["scale"]
    if c["residual"]:
        v = v + s["residual"].float()
    out["h"] = v.to(dt)
    if c["following"]:  # of the sum before it is rounded
        v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * (s["next"].float() + c["offset"])
        out["y"] = v.to(dt)
    if c["out8"] != "none":
        v = v.view(T, -1, c["out8_group"] or H)
        scale = v.abs().amax(2, keepdim=True) / QMAX[c["out8"]]
        q = v / scale
        q = torch.round(q) if c["out8"] == "int8" else q.to(torch.float8_e4m3fn).float()
        out["values"] = (q * scale).to(dt).view(T, H)
        out["scales"] = scale[:, :, 0]
    return out


# ------------------------------------------------------------------ the framework's calls

def _own_int8(s):
    from int4_grouped_gemm_router_amd import binding as B
    B.moe_project_int8(s["w"], s["w_scales"], s["x"], s["x_scales"], s["y"], s["c"]["T"], bias=s["bias"], ws=s["ws"])
    return {"y": s["y"]}


def _own_rope(s):
    from int4_grouped_gemm_router_amd import binding as B
    B.moe_rope(s["plan"], s["positions"], s["c"]["T"], s["q"], k=s["k"], q_out=s["q_out"], k_out=s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_linear(s):
    from int4_grouped_gemm_router_amd import binding as B
    c = s["c"]
    if c["step"]:
        B.moe_linear_attention_step(s["plan"], s["q"], s["k"], s["v"], s["decay"], s["o"], c["T"], state_in=s["pool"],
                                    slots_in=s["slots"], state_out=s["state"])
    else:
        B.moe_linear_attention(s["plan"], s["q"], s["k"], s["v"], s["decay"], s["o"], s["cu"], c["T"], state_in=s["pool"],
                               slots_in=s["slots"], state_out=s["state"], ws=s["ws"])
    return {"o": s["o"], "state": s["state"]}


def _own_gnorm(s):
    from int4_grouped_gemm_router_amd import binding as B
    c = s["c"]
    B.moe_gated_norm(s["plan"], s["x"], c["T"], weight=s["weight"], gate=s["gate"], channel_scale=s["channel"],
                     residual=s["residual"], next_weight=s["next"], h_out=s["h"], y=s["y"], q=s["q"], scales=s["q_scales"])
    out = {"h": s["h"]}
    if c["following"]:
        out["y"] = s["y"]
    if c["out8"] != "none":
        groups = s["q_scales"].shape[1]
        q = s["q"] if c["out8"] == "int8" else s["q"].float()
        torch.mul(q.view(c["T"], groups, -1), s["q_scales"][:, :, None], out=s["values"].view(c["T"], groups, -1))
        out["values"], out["scales"] = s["values"], s["q_scales"]
    return out


def run(state):
    if own:
        return {"int8": _own_int8, "rope": _own_rope, "linear": _own_linear, "gnorm": _own_gnorm}[state["c"]["op"]](state)
    return {"int8": _plain_int8, "rope": _plain_rope, "linear": _plain_linear, "gnorm": _plain_gnorm}[state["c"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(c):
    T = c["T"]
    if c["op"] == "int8":
        N, K, b = c["N"], c["K"], 4 if c["dtype"] == "f32" else 2
        return {"bytes": T * K + N * K + b * T * N + 4 * T + 4 * N * (1 + c["bias"]), "flops": 2 * T * N * K}
    if c["op"] == "rope":
        values = T * (c["q_heads"] + c["k_heads"]) * c["D"]
        return {"bytes": 2 * values * (4 if c["dtype"] == "f32" else 2) + 4 * T, "flops": 3 * values}
    if c["op"] == "linear":
        state = c["v_heads"] * c["dk"] * c["dv"]
        rows = T * (2 * (2 * c["k_heads"] * c["dk"] + 2 * c["v_heads"] * c["dv"]) + 4 * c["v_heads"] * c["per_token"])
        kept = c["seqs"] * (2.0 if c["step"] else 2.0 - c["fresh"])
        return {"bytes": rows + 4 * kept * state, "flops": 4 * T * state}
    H, b = c["H"], 4 if c["dtype"] == "f32" else 2
    values = T * H * (b * (2 + c["residual"] + c["following"] + (c["gate"] in ("silu", "sigmoid"))) + (c["out8"] != "none"))
    scales = 4 * T * (H // c["out8_group"] if c["out8_group"] else 1) if c["out8"] != "none" else 0
    return {"bytes": values + scales, "flops": 8 * T * H}


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3(v):
    """Nearest e4m3 value, ties to the even significand (|v| <= 448)."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp(min=-9))
    return torch.round(v / step) * step


def _exact_int8(s):
    y = torch.cat([s["x"].double() @ w.double().t() for w in s["w"].split(4096)], 1)
    y *= s["x_scales"].double()[:, None]
    y *= s["w_scales"].double()[None, :]
    return {"y": y if s["bias"] is None else y + s["bias"].double()}


def _exact_rope(s):
    c, out = s["c"], {}
    half = c["rot"] // 2
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        for i in range(half):
            at = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
            turn = torch.polar(torch.full_like(s["positions"], 1, dtype=torch.float64) * s["magnitude"],
                               s["positions"].double() * float(s["inv_freq"][i]))
            z = torch.complex(x[..., at[0]], x[..., at[1]]) * turn[:, None]
            y[..., at[0]], y[..., at[1]] = z.real, z.imag
        out[name] = y
    return out


def _exact_linear(s):
    c = s["c"]
    T, n, Hk, Hv, dk, dv = (c[k] for k in ("T", "seqs", "k_heads", "v_heads", "dk", "dv"))
    o = torch.empty((T, Hv, dv), dtype=torch.float64, device="cuda")
    state = torch.zeros((n, Hv, dk, dv), dtype=torch.float64, device="cuda")
    cu, slots = s["cu"].tolist(), s["slots"].tolist()
    for i in range(n):
        at = slice(cu[i], cu[i + 1])
        L = cu[i + 1] - cu[i]
        for h in range(Hv):
            q, k, v = s["q"][at, h * Hk // Hv].double(), s["k"][at, h * Hk // Hv].double(), s["v"][at, h].double()
            G = (s["decay"][at, h] if c["per_token"] else s["decay"][h].expand(L)).double().cumsum(0)
            S = s["pool"][slots[i], h].double() if slots[i] >= 0 else state[i, h]
            for a in range(0, L, 4096):  # queries of 4096 tokens against every key before them
                b = min(L, a + 4096)
                p = q[a:b] @ k[:b].t()
                p *= (G[a:b, None] - G[None, :b]).clamp(max=0).exp()
                o[cu[i] + a:cu[i] + b, h] = s["scale"] * (p.tril(a) @ v[:b] + G[a:b, None].exp() * (q[a:b] @ S))
            state[i, h] = G[-1].exp() * S + k.t() @ ((G[-1] - G).exp()[:, None] * v)
    return {"o": o, "state": state}


def _exact_gnorm(s):
    c, out = s["c"], {}
    T, H = c["T"], c["H"]
    m = s["x"].double()
    if c["after"]:
        parts = m.reshape(T, -1, c["group"] or H)
        rms = (parts.pow(2).sum(2, keepdim=True) / parts.shape[2] + EPS).sqrt()
        m = (parts / rms * (s["weight"].double() + c["offset"])).reshape(T, H)
    if c["gate"] != "none":
        z = s["gate"].double()
        m = m * (z * torch.sigmoid(z) if c["gate"] == "silu" else torch.sigmoid(z))
    v = m * c["scale"] * (s["channel"].double() if c["channel"] else 1.0)
    if c["residual"]:
        v = v + s["residual"].double()
    out["h"] = v
    if c["following"]:
        v = v / (v.pow(2).sum(1, keepdim=True) / H + EPS).sqrt() * (s["next"].double() + c["offset"])
        out["y"] = v
    if c["out8"] != "none":
        v = v.reshape(T, -1, c["out8_group"] or H)
        scale = v.abs().max(2, keepdim=True)[0] / QMAX[c["out8"]]
        q = (v / scale).round() if c["out8"] == "int8" else _e4m3(v / scale)
        out["values"] = (q * scale).reshape(T, H)
        out["scales"] = scale[:, :, 0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"int8": _exact_int8, "rope": _exact_rope, "linear": _exact_linear, "gnorm": _exact_gnorm}[case["op"]](s)
