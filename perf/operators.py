"""Cases for the operators around the int4 mixture-of-experts layer: the residual add + RMS norm
with an 8-bit output, the gated routing, and the packed int4 projection with low-rank adapters.

`run` computes an operator in elementary torch operations (`own` false) or through the binding
(`own` true); `exact` evaluates the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
QMAX = {"int8": 127.0, "e4m3": 448.0}


def _norm(name, T, H, dtype="bf16", weight="bf16", residual=True, y=True, out8="none", group=0, offset=0.0, pad=0):
    return {"name": name, "op": "norm", "T": T, "H": H, "dtype": dtype, "weight": weight, "residual": residual, "y": y,
            "out8": out8, "group": group, "offset": offset, "pad": pad}


def _route(name, T, E, k, score="softmax", bias=False, groups=1, keep=1, group_score="max", renorm=True, scale=1.0,
           block_m=32):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "bias": bias, "groups": groups,
            "keep": keep, "group_score": group_score, "renorm": renorm, "scale": scale, "block_m": block_m}


def _project(name, T, N, K, R, adapters, requests, plain_share=0.0, pad=0):
    return {"name": name, "op": "project", "T": T, "N": N, "K": K, "R": R, "adapters": adapters, "requests": requests,
            "plain_share": plain_share, "pad": pad}


def listed():
    return [
        # one decoded token entering the layer
        _norm("norm token", 1, 2048),
        # a prompt's rows for an 8-bit exchange between devices, one scale a row; nothing kept in bf16
        _norm("norm prompt int8", 512, 2048, y=False, out8="int8"),
        # a long prompt: bf16 rows for the router, e4m3 rows with a scale per 128 values for the experts
        _norm("norm long e4m3", 16384, 2048, out8="e4m3", group=128, offset=1.0),
        # an odd row length and row stride, fp16 activations under an fp32 weight, no residual
        _norm("norm odd f16", 777, 1537, dtype="f16", weight="f32", residual=False, pad=3),
        # one decoded token, sigmoid scores with a balance bias, 4 of 8 groups
        _route("route token", 1, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5),
        # a prompt of the 256-expert layer, softmax with a balance bias
        _route("route prompt", 512, 256, 8, "softmax", True),
        # a long prompt, sigmoid with groups
        _route("route long", 16384, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5),
        # an expert count that no wave divides, weights left as the softmax gives them
        _route("route odd", 2049, 60, 4, "softmax", renorm=False, block_m=16),
        # one decoded token with its adapter
        _project("project token", 1, 4096, 2048, 16, 8, 1),
        # one decoding step of 32 requests, each with an adapter of its own
        _project("project batch", 32, 4096, 2048, 16, 32, 32),
        # prompts of some requests, a part of them without an adapter, rows of a wider buffer
        _project("project prompts", 500, 2048, 2048, 32, 6, 9, plain_share=0.25, pad=64),
        # a long prefill chunk
        _project("project long", 4096, 4096, 2048, 16, 8, 5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "project"])
    if op == "norm":
        H = _log_int(rng, 128, 8192)
        group = rng.choice([0, 0, 32, 64, 128])
        if rng.random() < 0.75 or group:
            H = max(128, H // 128 * 128)
        T = _log_int(rng, 1, 16384 * 2048 // H)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if dtype == "f32":
            T = max(1, T // 2)
        out8 = rng.choice(["none", "int8", "e4m3"])
        y = out8 == "none" or rng.random() < 0.5
        c = _norm("", T, H, dtype, rng.choice([dtype, "f32"]), rng.random() < 0.7, y, out8, group if out8 != "none" else 0,
                  rng.choice([0.0, 1.0]), rng.choice([0, 0, 8, 3]))
    elif op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, 16 // groups), 256 // groups)
        keep = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(16, keep * (E // groups)))
        c = _route("", _log_int(rng, 1, 16384 * 8 // max(8, k)), E, k, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6,
                   groups, keep, rng.choice(["max", "top2"]), rng.random() < 0.7, rng.choice([1.0, 2.5]),
                   rng.choice([16, 32]))
    else:
        N = 64 * _log_int(rng, 8, 96)
        K = 128 * _log_int(rng, 4, 32)
        T = _log_int(rng, 1, min(4096, 4096 * 4096 * 2048 // (N * K)))
        R = rng.choice([8, 16, 24, 32, 64])
        adapters = _log_int(rng, 1, 48 if T < 1024 else 512 // R)
        c = _project("", T, N, K, R, adapters, _log_int(rng, 1, min(T, 64)),
                     rng.choice([0.0, 0.25]), rng.choice([0, 0, 8, 64]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _rows(g, T, width, pad, dtype, scale=1.0):
    """[T, width] of normal values in rows of width + pad."""
    full = torch.randn((T, width + pad), generator=g, device="cuda") * scale
    return full.to(dtype)[:, :width]


def _prepare_norm(c, g):
    dt = TYPES[c["dtype"]]
    T, H = c["T"], c["H"]
    s = {"c": c}
    # rows of different sizes, a few channels much larger than the rest, as a residual stream has them
    channel = torch.ones(H, device="cuda")
    channel[torch.randint(0, H, (max(1, H // 256),), generator=g, device="cuda")] = 20.0
    size = torch.exp(torch.randn((T, 1), generator=g, device="cuda") * 0.5)
    wide = torch.randn((T, H + c["pad"]), generator=g, device="cuda") * size
    wide[:, :H] *= channel
    s["x"] = _rows(g, T, H, c["pad"], dt)
    s["residual"] = wide.to(dt)[:, :H] if c["residual"] else None
    s["weight"] = (torch.rand(H, generator=g, device="cuda") * 0.5 + 0.75 - c["offset"]).to(TYPES[c["weight"]])
    if own:
        from int4_grouped_gemm_router_amd import binding as B
        s["plan"] = B.norm(H, dtype=dt, weight_dtype=TYPES[c["weight"]], eps=EPS, weight_offset=c["offset"],
                           out8={"none": B.OUT8_NONE, "int8": B.OUT8_INT8, "e4m3": B.OUT8_E4M3}[c["out8"]],
                           group=c["group"])
        new = lambda dtype: torch.empty((T, H + c["pad"]), dtype=dtype, device="cuda")[:, :H]  # noqa: E731
        s["h"] = new(dt) if c["residual"] else None
        s["y"] = new(dt) if c["y"] else None
        if c["out8"] != "none":
            s["q"] = torch.empty((T, H), dtype=torch.int8 if c["out8"] == "int8" else torch.float8_e4m3fn, device="cuda")
            s["scales"] = torch.empty((T, H // c["group"] if c["group"] else 1), dtype=torch.float32, device="cuda")
            if c["out8"] == "int8":
                s["values"] = torch.empty((T, H), dtype=dt, device="cuda")
    return s


def _prepare_route(c, g):
    T, E = c["T"], c["E"]
    # the layer's router: unit-variance rows times N(0, 0.02^2) weights over 2048 inputs, and experts that differ in
    # how often they are liked
    liked = torch.randn(E, generator=g, device="cuda") * 0.3
    s = {"c": c, "logits": torch.randn((T, E), generator=g, device="cuda") * 0.9 + liked}
    spread = 0.05 if c["score"] == "sigmoid" else 0.5 / E
    s["bias"] = (torch.rand(E, generator=g, device="cuda") * 2 - 1) * spread if c["bias"] else None
    if own:
        from int4_grouped_gemm_router_amd import binding as B
        s["gate"] = B.gate(E, top_k=c["k"], block_m=c["block_m"],
                           score=B.SCORE_SIGMOID if c["score"] == "sigmoid" else B.SCORE_SOFTMAX, n_groups=c["groups"],
                           topk_groups=c["keep"], group_score=B.GROUP_TOP2 if c["group_score"] == "top2" else B.GROUP_MAX,
                           renorm=c["renorm"], scale=c["scale"], balance_bias=s["bias"])
        s["out"] = B.RouteBuffers(s["gate"], T)
        s["ws"] = B.gate_workspace(s["gate"], T)
    return s


def _prepare_project(c, g):
    T, N, K, R, n = (c[k] for k in ("T", "N", "K", "R", "adapters"))
    q = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    scale = (torch.rand((N, K // 64), generator=g, device="cuda") * 0.015 + 0.005).to(torch.bfloat16)
    s = {"c": c, "x": _rows(g, T, K, c["pad"], torch.bfloat16), "q": q, "scale": scale, "bias": -8 * scale}
    s["A"] = (torch.randn((n, R, K), generator=g, device="cuda") / math.sqrt(K)).to(torch.bfloat16)
    s["B"] = (torch.randn((n, N, R), generator=g, device="cuda")).to(torch.bfloat16)
    s["ranks"] = torch.randint(max(1, R // 2), R + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    s["strength"] = torch.rand(n, generator=g, device="cuda") + 0.5
    # each request is a run of tokens; a run has one adapter, or none
    m = c["requests"]
    runs = torch.arange(T, device="cuda") * m // T
    of = torch.randperm(max(m, n), generator=g, device="cuda")[:m] % n
    of[torch.rand(m, generator=g, device="cuda") < c["plain_share"]] = -1
    s["adapter_of"] = of[runs].to(torch.int32)
    if own:
        from int4_grouped_gemm_router_amd import binding as B
        bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)[None]  # noqa: E731
        s["packed"] = torch.from_numpy(B.pack_int4_g64(q.cpu().numpy()[None], bits(scale), bits(s["bias"]))).cuda()
        s["adapters"] = B.Adapters(s["A"], s["B"], ranks=s["ranks"], scales=s["strength"])
        s["y"] = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        s["ws"] = B.project_workspace(N, K, T, s["adapters"])
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"norm": _prepare_norm, "route": _prepare_route, "project": _prepare_project}[case["op"]](case, g)


# ------------------------------------------------------------------ the plain forms

def _plain_norm(s):
    c, out = s["c"], {}
    h = s["x"]
    if c["residual"]:
        h = (h.float() + s["residual"].float()).to(h.dtype)
        out["h"] = h
    f = h.float()
    v = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * (s["weight"].float() + c["offset"])
    if c["y"]:
        out["y"] = v.to(h.dtype)
    if c["out8"] != "none":
        v = v.view(c["T"], -1, c["group"] or c["H"])
        scale = v.abs().amax(2, keepdim=True) / QMAX[c["out8"]]
        if c["out8"] == "int8":
            out["values"] = (torch.round(v / scale) * scale).to(h.dtype).view(c["T"], c["H"])
        else:
            out["q"] = (v / scale).to(torch.float8_e4m3fn).view(c["T"], c["H"])
        out["scales"] = scale[:, :, 0]
    return out


def _plain_route(s):
    c = s["c"]
    T, E, k, bm = c["T"], c["E"], c["k"], c["block_m"]
    l = s["logits"].double()  # ranks are decided between values that may be very close
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        score = torch.exp(l - l.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    key = score + s["bias"].double() if c["bias"] else score
    if c["groups"] > 1:
        per = key.view(T, c["groups"], -1)
        best = per.sort(dim=2, descending=True)[0]
        of_group = best[:, :, :2].sum(2) if c["group_score"] == "top2" else best[:, :, 0]
        kept = of_group.sort(dim=1, descending=True, stable=True)[1][:, : c["keep"]]
        mask = torch.zeros_like(of_group, dtype=torch.bool).scatter(1, kept, True)
        key = torch.where(mask[:, :, None], per, -math.inf).view(T, E)
    idx = key.sort(dim=1, descending=True, stable=True)[1][:, :k]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    flat = idx.reshape(-1)
    hist = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add(0, flat, torch.ones_like(flat))
    ends = hist.cumsum(0)
    perm = flat.sort(stable=True)[1]
    inv = torch.empty_like(perm).scatter(0, perm, torch.arange(T * k, device="cuda"))
    blocks = (hist + bm - 1) // bm
    block_ends = blocks.cumsum(0)
    j = torch.arange((T * k + bm - 1) // bm + E, device="cuda")
    e = torch.searchsorted(block_ends, j, right=True).clamp(max=E - 1)
    nth = j - (block_ends - blocks)[e]
    rows = torch.stack([e, (ends - hist)[e] + nth * bm, (hist[e] - nth * bm).clamp(max=bm)], 1)
    i32 = torch.int32
    return {"topk_idx": idx.to(i32), "topk_w": (w * c["scale"]).float(), "hist": hist.to(i32),
            "offsets": torch.cat([ends - hist, ends[-1:]]).to(i32), "perm": perm.to(i32), "inv_perm": inv.to(i32),
            "block_map": torch.where((j < block_ends[-1])[:, None], rows, -1).to(i32), "num_blocks": block_ends[-1:].to(i32)}


def _plain_project(s):
    c = s["c"]
    T, N, K, R, n = (c[k] for k in ("T", "N", "K", "R", "adapters"))
    w = s["q"].view(N, K // 64, 64).float() * s["scale"].float()[:, :, None] + s["bias"].float()[:, :, None]
    x = s["x"].float()
    y = x @ w.view(N, K).t()
    # every adapter on every token, and what is not the token's own put to zero
    z = (x @ s["A"].float().view(n * R, K).t()).view(T, n, R)
    factor = (s["adapter_of"][:, None] == torch.arange(n, device="cuda")).float() * s["strength"]
    held = (torch.arange(R, device="cuda") < s["ranks"][:, None]).float()
    z = z * factor[:, :, None] * held
    y = y + z.view(T, n * R) @ s["B"].float().transpose(1, 2).reshape(n * R, N)
    return {"y": y.to(torch.bfloat16)}


# ------------------------------------------------------------------ the framework's calls

def _own_norm(s):
    from int4_grouped_gemm_router_amd import binding as B
    c = s["c"]
    out = {}
    B.moe_add_rmsnorm(s["plan"], s["x"], s["weight"], c["T"], residual=s["residual"], h_out=s["h"], y=s["y"],
                      q=s.get("q"), scales=s.get("scales"))
    if c["residual"]:
        out["h"] = s["h"]
    if c["y"]:
        out["y"] = s["y"]
    if c["out8"] == "int8":
        groups = s["scales"].shape[1]
        torch.mul(s["q"].view(c["T"], groups, -1), s["scales"][:, :, None], out=s["values"].view(c["T"], groups, -1))
        out["values"] = s["values"]
    elif c["out8"] == "e4m3":
        out["q"] = s["q"]
    if c["out8"] != "none":
        out["scales"] = s["scales"]
    return out


def _own_route(s):
    from int4_grouped_gemm_router_amd import binding as B
    B.moe_route_gated(s["gate"], s["logits"], s["c"]["T"], s["out"], s["ws"])
    return {f: getattr(s["out"], f) for f in ("topk_idx", "topk_w", "hist", "offsets", "perm", "inv_perm", "block_map",
                                              "num_blocks")}


def _own_project(s):
    from int4_grouped_gemm_router_amd import binding as B
    c = s["c"]
    B.moe_project(s["packed"], c["N"], c["K"], s["x"], s["y"], c["T"], adapters=s["adapters"],
                  adapter_of=s["adapter_of"], ws=s["ws"])
    return {"y": s["y"]}


def run(state):
    if own:
        return {"norm": _own_norm, "route": _own_route, "project": _own_project}[state["c"]["op"]](state)
    return {"norm": _plain_norm, "route": _plain_route, "project": _plain_project}[state["c"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(c):
    if c["op"] == "norm":
        T, H, b = c["T"], c["H"], 4 if c["dtype"] == "f32" else 2
        values = T * H * (b * (1 + 2 * c["residual"] + c["y"]) + (c["out8"] != "none"))
        scales = 4 * T * (H // c["group"] if c["group"] else 1) if c["out8"] != "none" else 0
        return {"bytes": values + scales + H * (4 if c["weight"] == "f32" else 2), "flops": 6 * T * H}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 4 * T * E + 16 * T * k + 12 * (T * k // c["block_m"] + E), "flops": 8 * T * E}
    T, N, K, R = c["T"], c["N"], c["K"], c["R"]
    used = min(c["requests"], c["adapters"], T)
    return {"bytes": N * K // 2 + N * K // 16 + 2 * T * (K + N) + 2 * used * R * (K + N),
            "flops": 2 * T * N * K + 2 * T * R * (N + K)}


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3(v):
    """Nearest e4m3 value, ties to the even significand (|v| <= 448)."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp(min=-9))
    return torch.round(v / step) * step


def _exact_norm(s):
    c, out = s["c"], {}
    h = s["x"].double()
    if c["residual"]:
        h = (h + s["residual"].double()).to(s["x"].dtype).double()
        out["h"] = h
    v = h / (h.square().sum(1, keepdim=True) / c["H"] + EPS).sqrt() * (s["weight"].double() + c["offset"])
    if c["y"]:
        out["y"] = v
    if c["out8"] != "none":
        v = v.reshape(c["T"], -1, c["group"] or c["H"])
        scale = v.abs().max(2, keepdim=True)[0] / QMAX[c["out8"]]
        if c["out8"] == "int8":
            out["values"] = ((v / scale).round() * scale).reshape(c["T"], c["H"])
        else:
            out["q"] = _e4m3(v / scale).reshape(c["T"], c["H"])
        out["scales"] = scale[:, :, 0]
    return out


def _exact_route(s):
    c = s["c"]
    l = s["logits"].double()
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    key = score.clone() if s["bias"] is None else score + s["bias"].double()
    size = c["E"] // c["groups"]
    if c["groups"] > 1:
        per = key.view(c["T"], c["groups"], size)
        top = per.topk(min(size, 2 if c["group_score"] == "top2" else 1), 2)[0].sum(2)
        for _ in range(c["groups"] - c["keep"]):  # drop the weakest group, the later one of equals
            last = c["groups"] - 1 - top.flip(1).argmin(1)
            top[torch.arange(c["T"], device=top.device), last] = math.inf
            per[torch.arange(c["T"], device=top.device), last] = -math.inf
    chosen = []
    for _ in range(c["k"]):
        best = key.argmax(1, keepdim=True)
        chosen.append(score.gather(1, best))
        key.scatter_(1, best, -math.inf)
    w = torch.cat(chosen, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"topk_idx": None, "topk_w": w * c["scale"], "hist": None, "offsets": None, "perm": None, "inv_perm": None,
            "block_map": None, "num_blocks": None}


def _exact_project(s):
    c = s["c"]
    x = s["x"].double()
    groups = [t.double().repeat_interleave(64, 1) for t in (s["scale"], s["bias"])]
    y = x @ (s["q"].double() * groups[0] + groups[1]).t()
    for a in range(c["adapters"]):
        at = (s["adapter_of"] == a).nonzero()[:, 0]
        r = int(s["ranks"][a])
        if len(at):
            y[at] += s["strength"][a].double() * (x[at] @ s["A"][a, :r].double().t() @ s["B"][a, :, :r].double().t())
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "project": _exact_project}[case["op"]](s)
