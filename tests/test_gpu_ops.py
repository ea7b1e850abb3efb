"""GPU parity of the operators around the layer: residual add + RMS norm with 8-bit outputs, gated
routing (alone and in the layer), the int4 projection with adapters, and a run of them together.

Every result is compared with a plain implementation in 64 bits (ops_ref.py); the tolerances there are
bounds derived from the number formats."""
import numpy as np
import pytest
import torch

import oracle
from int4_grouped_gemm_router_amd import binding as B
from int4_grouped_gemm_router_amd import synth

from ops_ref import U32, block_map_ref, gate_ref, half_step, norm_ref, norm_rel, project_ref
from parity import check_layer, check_route_meta

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GUARD = 0x5A


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def _wide(t, pad, rows=0, fill=7.0):
    """A device copy of a CPU [T, W] tensor as a view of [T + rows, W + pad] filled with `fill`."""
    full = torch.full((t.shape[0] + rows, t.shape[1] + pad), fill, dtype=t.dtype)
    full[:t.shape[0], :t.shape[1]] = t
    full = full.cuda()
    return full[:t.shape[0], :t.shape[1]], full


def _behind(full, T, W, fill=7.0):
    """Whether everything outside the first [T, W] still holds `fill`."""
    f = full.float().cpu()
    return bool((f[T:] == fill).all() and (f[:T, W:] == fill).all())


def _graph_us(f, n=20):
    for _ in range(3):
        f()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(n):
            f()
    best = float("inf")
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / n * 1e3)
    return best


# ------------------------------------------------------------------ residual add + RMS norm

def _norm_case(T, H, dtype="bf16", weight=None, residual=True, y=True, out8=B.OUT8_NONE, group=0, offset=0.0, pad=0,
               seed=0, x=None, eps=1e-6):
    g = torch.Generator().manual_seed(seed + 31 * T + H)
    dt = DT[dtype]
    if x is None:
        x = torch.randn((T, H), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    x = x.to(dt)
    res = (torch.randn((T, H), generator=g) * 2).to(dt) if residual else None
    w = (torch.rand(H, generator=g) + 0.5 - offset).to(DT[weight or dtype])
    n = B.norm(H, dtype=dt, weight_dtype=w.dtype, eps=eps, weight_offset=offset, out8=out8, group=group)
    xv, xf = _wide(x, pad, 1)
    rv = _wide(res, pad, 1)[0] if residual else None
    hv, hf = _wide(torch.zeros_like(x), pad, 2)
    yv, yf = _wide(torch.zeros_like(x), pad, 2)
    q = s = qf = None
    G = H // group if group else 1
    if out8:
        q, qf = _wide(torch.zeros((T, H), dtype=torch.uint8), pad, 2, GUARD)
        s = torch.full((T + 1, G), -1.0, device="cuda")
    B.moe_add_rmsnorm(n, xv, w.cuda(), T, residual=rv, h_out=hv if residual else None, y=yv if y else None, q=q,
                      scales=s)
    torch.cuda.synchronize()
    h, v = norm_ref(x, res, w, eps, offset)
    if residual:
        assert torch.equal(hv.cpu(), h)
        assert _behind(hf, T, H)
    rel = norm_rel(H)
    if y:
        err = (yv.cpu().double() - v).abs()
        tol = half_step(dt, v) * (1 + rel) + rel * v.abs()
        assert (err <= tol).all(), f"y: {(err / tol).max():.3f} of its bound"
        assert _behind(yf, T, H)
    if out8:
        Q = 127.0 if out8 == B.OUT8_INT8 else 448.0
        vg = v.reshape(T, G, -1)
        sref = vg.abs().amax(2) / Q
        sc = s.cpu().double()
        assert ((sc[:T] - sref).abs() <= sref * (rel + 2 * U32)).all()
        assert (sc[T:] == -1).all()
        assert _behind(qf, T, H, GUARD)
        want = torch.where(sref[:, :, None] > 0, vg / sref[:, :, None].clamp(min=1e-300), torch.zeros_like(vg))
        off = want.abs() * (2 * rel + 4 * U32)  # of v and of the scale, and of the quotient
        if out8 == B.OUT8_INT8:
            got = q.cpu().view(torch.int8).double().reshape(vg.shape)
            assert (got.abs() <= 127).all()
            step = 0.5
        else:
            got = q.cpu().contiguous().view(torch.float8_e4m3fn).double().reshape(vg.shape)
            step = (want.abs() * 2.0 ** -4).clamp(min=2.0 ** -10)  # half a step: 2^-4 relative, 2^-10 below 2^-6
        assert ((got - want).abs() <= step + off).all()
    return xv, xf


NORM_CASES = [
    # one row to many, the layer's hidden size and others
    dict(T=1, H=2048), dict(T=3, H=2048), dict(T=64, H=2048), dict(T=700, H=2048, residual=False),
    dict(T=5, H=1), dict(T=5, H=2), dict(T=4, H=7), dict(T=9, H=63), dict(T=9, H=65), dict(T=3, H=511), dict(T=3, H=1537),
    dict(T=2, H=2056), dict(T=2, H=4096), dict(T=2, H=5000), dict(T=2, H=8192), dict(T=2, H=8200), dict(T=2, H=16384),
    dict(T=2, H=16383),
    # types
    dict(T=33, H=1024, dtype="f16"), dict(T=33, H=1024, dtype="f32"), dict(T=33, H=1537, dtype="f16", weight="f32"),
    dict(T=33, H=1024, weight="f32", offset=1.0), dict(T=17, H=130, dtype="f32"), dict(T=2, H=16384, dtype="f32"),
    # strides that break the alignment of rows
    dict(T=33, H=1024, pad=8), dict(T=33, H=1024, pad=1), dict(T=33, H=1024, pad=4), dict(T=33, H=1024, pad=3, dtype="f32"),
    # 8-bit outputs
    dict(T=1, H=2048, out8=B.OUT8_INT8), dict(T=300, H=2048, out8=B.OUT8_INT8, y=False),
    dict(T=300, H=2048, out8=B.OUT8_E4M3, group=128, offset=1.0), dict(T=65, H=2048, out8=B.OUT8_E4M3),
    dict(T=65, H=2048, out8=B.OUT8_INT8, group=32), dict(T=65, H=2048, out8=B.OUT8_E4M3, group=64, dtype="f16"),
    dict(T=65, H=512, out8=B.OUT8_INT8, group=256, dtype="f32"), dict(T=7, H=32, out8=B.OUT8_INT8, group=32),
    dict(T=7, H=96, out8=B.OUT8_E4M3, group=32, pad=1), dict(T=7, H=384, out8=B.OUT8_INT8, group=128, pad=3),
    dict(T=7, H=1000, out8=B.OUT8_INT8), dict(T=7, H=333, out8=B.OUT8_E4M3), dict(T=4, H=16384, out8=B.OUT8_INT8, group=256),
    dict(T=4, H=9000, out8=B.OUT8_E4M3), dict(T=4, H=768, out8=B.OUT8_INT8, group=256, pad=2),
    dict(T=4, H=16384, out8=B.OUT8_E4M3, group=128, pad=5), dict(T=2000, H=64, out8=B.OUT8_INT8, group=32),
]


@pytest.mark.parametrize("c", NORM_CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_norm_matches_64_bits(c):
    _norm_case(**c)


@pytest.mark.parametrize("T,H", [(70001, 64), (20001, 500), (17003, 1024), (4999, 2048), (6001, 2056), (4100, 4104)])
@pytest.mark.parametrize("out8,group", [(B.OUT8_INT8, 0), (B.OUT8_E4M3, 32)])
def test_norm_blocks_take_rows_in_turn(T, H, out8, group):
    # more rows than the grid holds at once, for each number of threads a row
    _norm_case(T, H, out8=out8, group=group if H % 32 == 0 else 0)


@pytest.mark.parametrize("out8,group", [(B.OUT8_INT8, 0), (B.OUT8_E4M3, 64)])
def test_norm_zero_and_tiny_rows(out8, group):
    # rows of zeros (scale 0, q 0), rows far below eps, and one large value among zeros
    x = torch.zeros(4, 256)
    x[1] = 1e-20
    x[2, 77] = -300.0
    x[3, 64:128] = torch.linspace(-1, 1, 64)
    _norm_case(4, 256, residual=False, out8=out8, group=group, x=x)
    _norm_case(4, 256, dtype="f32", residual=False, out8=out8, group=group, x=x)


def test_norm_int8_ties_of_wide_products():
    # fp16 rows times fp16 weights have up to 22 bits and Q seven more: in a group of weight w with the largest value
    # 254 w, (2 k + 1) w is exactly k + 1/2 steps and goes to the even one, whatever w is (the row's factor cancels)
    H, group = 16384, 128
    x = torch.cat([torch.arange(1, 254, 2), torch.tensor([254])]).repeat(H // group)[None].to(torch.float16)
    w = ((1025 + 8 * torch.arange(H // group)) / 1024).repeat_interleave(group).to(torch.float16)
    q = torch.zeros((1, H), dtype=torch.int8, device="cuda")
    s = torch.zeros((1, H // group), device="cuda")
    B.moe_add_rmsnorm(B.norm(H, dtype=torch.float16, out8=B.OUT8_INT8, group=group), x.cuda(), w.cuda(), 1, q=q, scales=s)
    assert torch.equal(q.cpu().double(), torch.round(x.double() / 2))      # (torch rounds ties to even)


def test_norm_nan_and_infinity_stay_in_their_row():
    T, H = 4, 512
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    w = torch.ones(H, dtype=torch.bfloat16)
    for out8 in (B.OUT8_INT8, B.OUT8_E4M3):
        n = B.norm(H, out8=out8, group=128)
        y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        q = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
        s = torch.zeros(T, H // 128, device="cuda")
        B.moe_add_rmsnorm(n, x.cuda(), w.cuda(), T, y=y, q=q, scales=s)
        y, s, q = y.float().cpu(), s.cpu(), q.cpu()
        assert y[1].isnan().all() and s[1].isnan().all()
        assert y[2, 200].isnan() and (y[2, :200] == 0).all() and s[2, 1].isnan()
        assert y[[0, 3]].isfinite().all() and s[[0, 3]].isfinite().all()
        assert (q[1] == (0 if out8 == B.OUT8_INT8 else 0x7F)).all() or out8 == B.OUT8_E4M3
        if out8 == B.OUT8_E4M3:
            assert q[1].view(torch.float8_e4m3fn).float().isnan().all()


@pytest.mark.parametrize("H", [2048, 1537])
def test_norm_in_place(H):
    # h over the residual and y over x, and y over h
    g = torch.Generator().manual_seed(H)
    x, r = (torch.randn(9, H, generator=g).to(torch.bfloat16) for _ in range(2))
    w = torch.rand(H, generator=g).to(torch.bfloat16).cuda()
    n = B.norm(H)
    h0, y0 = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    B.moe_add_rmsnorm(n, x.cuda(), w, 9, residual=r.cuda(), h_out=h0, y=y0)
    xd, rd = x.cuda(), r.cuda()
    B.moe_add_rmsnorm(n, xd, w, 9, residual=rd, h_out=rd, y=xd)
    assert torch.equal(rd, h0) and torch.equal(xd, y0)
    xd, rd = x.cuda(), r.cuda()
    B.moe_add_rmsnorm(n, xd, w, 9, residual=rd, h_out=rd, y=rd)
    assert torch.equal(rd, y0)
    xd = x.cuda()
    B.moe_add_rmsnorm(n, xd, w, 9, residual=r.cuda(), h_out=xd)   # the sum alone
    assert torch.equal(xd, h0)


def test_one_row_of_any_stride():
    # the last token of a prompt [1, S, H]: its row stride, S H, is more than 2^20; and a stride that is no multiple of 8
    H, N, S = 2048, 64, 600
    prompt = torch.randn((1, S, H), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    w, m = torch.ones(H, dtype=torch.bfloat16, device="cuda"), _Matrix(N, H)
    far, near = prompt[:, -1], prompt[:, -1].clone()
    assert far.stride(0) > 1 << 20
    odd = torch.zeros(H + 1, dtype=torch.bfloat16, device="cuda").as_strided((1, H), (H + 1, 1))
    odd.copy_(near)
    want, wide = torch.empty_like(near), torch.empty((1, N), dtype=torch.bfloat16, device="cuda")
    B.moe_add_rmsnorm(B.norm(H), near, w, 1, y=want)
    B.moe_project(m.blob, N, H, near, wide, 1, ws=B.project_workspace(N, H, 1))
    for x in (far, odd):
        got, p = torch.empty_like(near), torch.empty_like(wide)
        B.moe_project(m.blob, N, H, x, p, 1, ws=B.project_workspace(N, H, 1))
        B.moe_add_rmsnorm(B.norm(H), x, w, 1, y=got)
        B.moe_add_rmsnorm(B.norm(H), x, w, 1, y=x.as_strided((1, H), (H, 1), x.storage_offset()))   # in place
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(x, want) and torch.equal(p, wide)


# ------------------------------------------------------------------ gated routing

SCORES = {"softmax": B.SCORE_SOFTMAX, "sigmoid": B.SCORE_SIGMOID}
GROUP = {"max": B.GROUP_MAX, "top2": B.GROUP_TOP2}


def _logits(rng, T, E, kind):
    l = (rng.normal(size=(T, E)) * 1.3).astype(np.float32)
    if kind == "ties":
        l = np.round(l * 2) / 2
        l[l == 0] = rng.choice(np.array([0.0, -0.0], np.float32), size=int((l == 0).sum()))
    if kind == "masked":
        l[rng.random((T, E)) < 0.4] = -np.inf
        l[rng.random((T, E)) < 0.05] = np.nan
        l[0] = -np.inf                       # rows with nothing left
        l[-1] = np.nan
        if T > 4:
            l[1, :] = -np.inf
            l[1, E // 2] = 0.5               # one expert left
            l[2, E - 1] = np.inf
            l[3, [0, E - 1]] = np.inf
            l[4, : E // 2] = np.finfo(np.float32).min
    return l.astype(np.float32)


def _run_gate(l, top_k, score, n_groups=1, topk_groups=1, group_score="max", renorm=True, scale=1.0, bias=None,
              block_m=32, stream=None):
    T, E = l.shape
    bt = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    g = B.gate(E, top_k, block_m, SCORES[score], n_groups, topk_groups, GROUP[group_score], renorm, scale, bt)
    out = B.RouteBuffers(g, T)
    ws = B.gate_workspace(g, T)
    ws.fill_(0xA5)
    B.moe_route_gated(g, torch.from_numpy(l).cuda(), T, out, ws, stream)
    torch.cuda.synchronize()
    return out.to_numpy()


def _check_gate(l, meta, top_k, block_m=32, **kw):
    T, E = l.shape
    idx, w = gate_ref(l, top_k, **kw)
    assert np.array_equal(meta["topk_idx"], idx)
    # one fp32 rounding of a value computed in 64 bits, or fp32 exponentials, at most 16 of them summed:
    # 2 ulp each, 5 additions, a division and the scale
    tol = np.abs(w) * (16 * U32) + 1e-37
    assert (np.abs(meta["topk_w"] - w) <= tol).all(), f"weights: {(np.abs(meta['topk_w'] - w) / tol).max():.2f}"
    check_route_meta(meta, idx, E, top_k, block_m)
    assert np.array_equal(meta["block_map"], block_map_ref(idx, E, block_m))


GATES = [
    dict(top_k=8, score="softmax"), dict(top_k=8, score="softmax", renorm=False, scale=2.5),
    dict(top_k=8, score="sigmoid", bias="small"), dict(top_k=6, score="sigmoid", bias="wide", renorm=False),
    dict(top_k=8, score="sigmoid", bias="small", n_groups=8, topk_groups=4, group_score="top2", scale=2.5),
    dict(top_k=6, score="softmax", n_groups=8, topk_groups=3, group_score="max", renorm=False, scale=16.0),
    dict(top_k=1, score="sigmoid"), dict(top_k=16, score="softmax", bias="small", block_m=16),
    dict(top_k=4, score="softmax", n_groups=64, topk_groups=9, group_score="top2"),
    dict(top_k=2, score="sigmoid", n_groups=2, topk_groups=1, group_score="top2", bias="nan"),
]


def _ids(c):
    return "-".join(f"{k}{v}" for k, v in c.items())


@pytest.mark.parametrize("kind", ["plain", "ties", "masked"])
@pytest.mark.parametrize("c", GATES, ids=_ids)
def test_gate_matches_64_bits(c, kind):
    c = dict(c)
    for T, E in ((1, 256), (7, 64), (129, 256), (300, 192)):
        if E % c.get("n_groups", 1):
            continue
        if c.get("topk_groups", 1) * (E // c.get("n_groups", 1)) < c["top_k"]:
            continue
        rng = np.random.default_rng(T + E + len(kind))
        kw = dict(c)
        kind_of_bias = kw.pop("bias", None)
        if kind_of_bias:
            kw["bias"] = rng.uniform(-1, 1, E).astype(np.float32) * {"small": 0.05, "wide": 3.0, "nan": 0.3}[kind_of_bias]
            if kind_of_bias == "nan":
                kw["bias"][[1, E // 2]] = np.nan, -np.inf
        l = _logits(rng, T, E, kind)
        _check_gate(l, _run_gate(l, **kw), **kw)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 2, 2), (33, 3, 1), (40, 60, 4), (2049, 60, 4), (17, 65, 16), (100, 255, 8),
                                   (9, 16, 16), (1000, 10, 3), (4097, 256, 8), (127, 256, 8), (128, 256, 8), (513, 128, 2)])
def test_gate_odd_sizes(T, E, k):
    rng = np.random.default_rng(T * 3 + E)
    for score in ("softmax", "sigmoid"):
        kw = dict(top_k=k, score=score, bias=rng.uniform(-0.1, 0.1, E).astype(np.float32), renorm=score == "sigmoid")
        l = _logits(rng, T, E, "plain")
        _check_gate(l, _run_gate(l, block_m=16, **kw), block_m=16, **kw)


@pytest.mark.parametrize("T,E,k", [(65537, 24, 3), (70001, 200, 1), (140000, 8, 2)])
def test_gate_many_tokens(T, E, k):
    # several pieces of tokens for each block of the scatter
    rng = np.random.default_rng(T)
    l = _logits(rng, T, E, "plain")
    _check_gate(l, _run_gate(l, top_k=k, score="softmax"), top_k=k, score="softmax")


def test_gate_keys_closer_than_fp32():
    # score + bias differ by less than an fp32 exponential errs: the bias of expert e makes its key the
    # same as its neighbour's up to the bias's own rounding, so only 64 bits tell them apart
    rng = np.random.default_rng(3)
    for score in ("softmax", "sigmoid"):
        for T in (1, 64):
            l = rng.normal(size=(T, 64)).astype(np.float32)
            ld = l[0].astype(np.float64)
            s = 1 / (1 + np.exp(-ld)) if score == "sigmoid" else np.exp(ld - ld.max()) / np.exp(ld - ld.max()).sum()
            bias = (0.75 - s).astype(np.float32)
            l[:] = l[0]
            kw = dict(top_k=8, score=score, bias=bias)
            _check_gate(l, _run_gate(l, **kw), **kw)
            kw.update(n_groups=8, topk_groups=4, group_score="top2")
            _check_gate(l, _run_gate(l, **kw), **kw)


@pytest.mark.parametrize("equal", [2, 9, 63, 64, 65, 100, 256])
def test_gate_many_equal_keys(equal):
    # `equal` experts share the largest key; with a bias, with groups and without
    rng = np.random.default_rng(equal)
    for T in (1, 70):
        l = rng.normal(size=(T, 256)).astype(np.float32)
        for t in range(T):
            l[t, rng.permutation(256)[:equal]] = 5.0
        for kw in (dict(score="softmax"), dict(score="sigmoid", bias=np.full(256, 0.25, np.float32)),
                   dict(score="sigmoid", n_groups=8, topk_groups=4, group_score="top2"),
                   dict(score="softmax", n_groups=32, topk_groups=9)):
            _check_gate(l, _run_gate(l, top_k=8, **kw), top_k=8, **kw)


def _mask_bias(rng, E, kind, share):
    """Balance biases in which a share of the experts is masked in one of several ways."""
    bias = rng.uniform(-0.05, 0.05, E).astype(np.float32)
    far = {"inf": [-np.inf], "nan": [np.nan], "1e4": [-1e4], "1e9": [-1e9], "max": [-3e38], "2": [-2.0, -1.0],
           "mixed": [-np.inf, np.nan, -9.0, -1e3, -1e9, -3e38], "above": [1e9, 50.0], "plus": [np.inf]}[kind]
    at = rng.permutation(E)[: max(1, int(E * share))]
    bias[at] = rng.choice(np.array(far, np.float32), size=len(at))
    return bias


@pytest.mark.parametrize("share", [0.0, 0.3, 0.8, 0.985])
@pytest.mark.parametrize("kind", ["inf", "nan", "1e4", "1e9", "max", "2", "mixed", "above", "plus"])
def test_gate_biases_that_mask_experts(kind, share):
    # one expert, a part of them, so many that some groups have none left, and all but a few
    for T, E in ((3, 256), (70, 256), (40, 128), (40, 64)):
        rng = np.random.default_rng(T + E + int(100 * share))
        bias = _mask_bias(rng, E, kind, share)
        for score in ("softmax", "sigmoid"):
            l = _logits(rng, T, E, "plain")
            for kw in (dict(), dict(n_groups=8, topk_groups=4, group_score="top2"),
                       dict(n_groups=16, topk_groups=5, group_score="max", renorm=False), dict(n_groups=32, topk_groups=9)):
                kw = dict(top_k=8, score=score, bias=bias, **kw)
                if kw.get("topk_groups", 1) * (E // kw.get("n_groups", 1)) >= 8:
                    _check_gate(l, _run_gate(l, **kw), **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_large_biases_of_one_size(score):
    # keys whose bias hides most of the score's bits, or all of them
    for offset in (5.0, 300.0, 1e6, -1e6, -1e20, 1e29, -1e31):
        rng = np.random.default_rng(int(abs(offset)) % 1000)
        l = _logits(rng, 50, 256, "plain")
        bias = (rng.uniform(-0.05, 0.05, 256) + offset).astype(np.float32)
        for kw in (dict(), dict(n_groups=8, topk_groups=4, group_score="top2")):
            kw = dict(top_k=8, score=score, bias=bias, **kw)
            _check_gate(l, _run_gate(l, **kw), **kw)


@pytest.mark.parametrize("masked", [-np.inf, np.nan, -1e4, -1e9])
def test_gate_masking_an_expert_costs_no_decisions_in_64_bits(masked):
    # decided in 64 bits, every token of a call, the routing took three times as long
    T, E = 16384, 256
    rng = np.random.default_rng(8)
    logits = torch.from_numpy(_logits(rng, T, E, "plain")).cuda()
    us = []
    for value in (None, masked):
        bias = rng.uniform(-0.05, 0.05, E).astype(np.float32)
        if value is not None:
            bias[E // 3] = value
        g = B.gate(E, 8, score=B.SCORE_SIGMOID, n_groups=8, topk_groups=4, group_score=B.GROUP_TOP2,
                   balance_bias=torch.from_numpy(bias).cuda())
        out, ws = B.RouteBuffers(g, T), B.gate_workspace(g, T)
        us.append(_graph_us(lambda: B.moe_route_gated(g, logits, T, out, ws)))
    assert us[1] < 1.6 * us[0], us


def test_gate_softmax_agrees_with_moe_route():
    rng = np.random.default_rng(12)
    T, E = 1000, 256
    l = synth.random_logits(rng, T, E, ties=50)
    meta = _run_gate(l, top_k=8, score="softmax")
    d = B.dims(2048, 512)
    out = B.RouteBuffers(d, T)
    B.moe_route(d, torch.from_numpy(l).cuda(), T, out, B.workspace(d, T, B.MODE_ROUTE))
    torch.cuda.synchronize()
    ref = out.to_numpy()
    for f in ("topk_idx", "hist", "offsets", "perm", "inv_perm", "block_map", "num_blocks"):
        assert np.array_equal(meta[f], ref[f]), f
    assert np.allclose(meta["topk_w"], ref["topk_w"], rtol=1e-6, atol=0)


# ------------------------------------------------------------------ the gated layer

def _layer_ref(x, w, idx, wsel):
    """y of the layer for given experts and weights, from the oracle's expert."""
    def expert(e, row):
        return oracle.expert_ffn(row, *[(w.q[m][e], w.scale[m][e], w.bias[m][e]) for m in ("gate", "up", "down")])
    y = np.empty((x.shape[0], w.H))
    for t in range(x.shape[0]):
        y[t] = expert(w.E, x[t])
        for e, v in zip(idx[t], wsel[t]):
            y[t] += v * expert(int(e), x[t])
    return y


GATE_DSV = dict(top_k=8, score="sigmoid", n_groups=8, topk_groups=4, group_score="top2", scale=2.5)


@pytest.mark.parametrize("T,chunk", [(1, 0), (3, 0), (4, 0), (33, 0), (50, 16)])
def test_gated_layer(T, chunk):
    rng = np.random.default_rng(60 + T)
    _, w, _ = synth.generate("tiny_t32", with_x=False)
    dw = B.DeviceWeights.from_logical(w)
    x = synth.make_x(rng, T, w.H)
    bias = rng.uniform(-0.05, 0.05, w.E).astype(np.float32)
    g = B.gate(w.E, 8, score=B.SCORE_SIGMOID, n_groups=8, topk_groups=4, group_score=B.GROUP_TOP2, scale=2.5,
               balance_bias=torch.from_numpy(bias).cuda())
    d = dw.dims
    runs = [("prefill", B.moe_prefill_layer_gated, B.MODE_PREFILL)]
    if T <= 4:
        runs.append(("decode", B.moe_decode_layer_gated, B.MODE_DECODE))
    for name, f, mode in runs:
        Tc = chunk or T
        last = T - (T - 1) // Tc * Tc
        y = torch.empty((T, w.H), dtype=torch.int16, device="cuda")
        logits = torch.empty((T, w.E), device="cuda")
        ro = B.RouteBuffers(d, last)
        args = [d, g, dw, torch.from_numpy(x).cuda(), y, T] + ([chunk] if mode == B.MODE_PREFILL else [])
        f(*args, logits_out=logits, route_out=ro, ws=B.workspace(d, Tc, mode))
        torch.cuda.synchronize()
        idx, wsel = gate_ref(logits.cpu().numpy(), bias=bias, **GATE_DSV)
        meta = ro.to_numpy()
        assert np.array_equal(meta["topk_idx"], idx[T - last:]), name
        check_route_meta(meta, idx[T - last:], w.E, 8, 32)
        ref = _layer_ref(x, w, idx, wsel)
        got = synth.bf16_bits_to_f32(y.cpu().numpy().view(np.uint16)).astype(np.float64)
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= 5e-3, f"{name}: {rel}"     # the layer's own bar


def _check_gated_layer(w, dw, d, T, mode, tokens=None):
    """One call of the layer with a gate; y of `tokens` (all by default) against the oracle's experts."""
    rng = np.random.default_rng(900 + T + w.H)
    x = synth.make_x(rng, T, w.H)
    bias = rng.uniform(-0.05, 0.05, w.E).astype(np.float32)
    bias[5] = -np.inf                                          # an expert that is never selected
    g = B.gate(w.E, 8, score=B.SCORE_SIGMOID, n_groups=8, topk_groups=4, group_score=B.GROUP_TOP2, scale=2.5,
               balance_bias=torch.from_numpy(bias).cuda())
    y = torch.full((T + 1, w.H), 0x5A5A, dtype=torch.int16, device="cuda")
    logits, ro = torch.empty((T, w.E), device="cuda"), B.RouteBuffers(d, T)
    f = B.moe_decode_layer_gated if mode == B.MODE_DECODE else B.moe_prefill_layer_gated
    ws = B.workspace(d, T, mode)
    ws.fill_(0xA5)
    f(d, g, dw, torch.from_numpy(x).cuda(), y, T, logits_out=logits, route_out=ro, ws=ws)
    torch.cuda.synchronize()
    assert (y[T] == 0x5A5A).all()
    idx, wsel = gate_ref(logits.cpu().numpy(), bias=bias, **GATE_DSV)
    meta = ro.to_numpy()
    assert np.array_equal(meta["topk_idx"], idx)
    assert (np.abs(meta["topk_w"] - wsel) <= np.abs(wsel) * (16 * U32) + 1e-37).all()
    check_route_meta(meta, idx, w.E, 8, 32)
    at = np.arange(T) if tokens is None else np.linspace(0, T - 1, tokens).astype(int)
    ref = _layer_ref(x[at], w, idx[at], wsel[at])
    got = synth.bf16_bits_to_f32(y[:T].cpu().numpy().view(np.uint16)).astype(np.float64)[at]
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert rel <= 5e-3, rel                                    # the layer's own bar


def test_gated_layer_real_size():
    _, w, _ = synth.generate("prefill_t512", with_x=False)
    dw = B.DeviceWeights.from_logical(w)
    for T in (1, 2, 3, 4):
        _check_gated_layer(w, dw, dw.dims, T, B.MODE_DECODE)
    _check_gated_layer(w, dw, dw.dims, 2, B.MODE_PREFILL)
    for gemm in (B.GEMM_EXACT, B.GEMM_WIDE):
        _check_gated_layer(w, dw, B.dims(w.H, w.I, w.E, gemm=gemm), 512, B.MODE_PREFILL, tokens=16)


@pytest.mark.parametrize("H,I,E", [(256, 128, 64), (1024, 256, 128), (4096, 128, 64), (768, 384, 192)])
def test_gated_layer_other_sizes(H, I, E):
    w = synth.make_weights(np.random.default_rng(H), H, I, E)
    dw = B.DeviceWeights.from_logical(w)
    for T in (1, 2, 4):
        _check_gated_layer(w, dw, dw.dims, T, B.MODE_DECODE)
    _check_gated_layer(w, dw, dw.dims, 37, B.MODE_PREFILL)


@pytest.mark.parametrize("T", [1, 4, 33])
def test_gated_layer_without_its_optional_outputs(T):
    _, w, _ = synth.generate("tiny_t32", with_x=False)
    dw, d = B.DeviceWeights.from_logical(w), B.dims(w.H, w.I, w.E)
    x = torch.from_numpy(synth.make_x(np.random.default_rng(T), T, w.H)).cuda()
    g = B.gate(w.E, 8, score=B.SCORE_SIGMOID)
    for f, mode in ((B.moe_prefill_layer_gated, B.MODE_PREFILL), (B.moe_decode_layer_gated, B.MODE_DECODE)):
        if mode == B.MODE_DECODE and T > 4:
            continue
        y = [torch.empty((T, w.H), dtype=torch.int16, device="cuda") for _ in range(2)]
        f(d, g, dw, x, y[0], T, ws=B.workspace(d, T, mode))
        f(d, g, dw, x, y[1], T, logits_out=torch.empty((T, w.E), device="cuda"), route_out=B.RouteBuffers(d, T),
          ws=B.workspace(d, T, mode))
        assert torch.equal(*y)


@pytest.mark.parametrize("E", [256, 60])
def test_gate_logits_and_biases_at_any_word(E):
    rng, T = np.random.default_rng(E), 100
    l, bias = _logits(rng, T, E, "plain"), rng.uniform(-0.05, 0.05, E).astype(np.float32)
    want = _run_gate(l, 8, "sigmoid", bias=bias)
    for lo, bo in ((1, 0), (0, 3), (2, 1)):
        lt = torch.zeros(T * E + 3, device="cuda")[lo : lo + T * E].view(T, E)
        bt = torch.zeros(E + 3, device="cuda")[bo : bo + E]
        lt.copy_(torch.from_numpy(l))
        bt.copy_(torch.from_numpy(bias))
        g = B.gate(E, 8, score=B.SCORE_SIGMOID, balance_bias=bt)
        out = B.RouteBuffers(g, T)
        B.moe_route_gated(g, lt, T, out, B.gate_workspace(g, T))
        got = out.to_numpy()
        for name in want:
            assert np.array_equal(got[name], want[name]), name


def test_gate_binding_checks_tensors():
    _, w, _ = synth.generate("tiny_t32", with_x=False)
    dw, T = B.DeviceWeights.from_logical(w), 2
    x = torch.zeros((T, w.H), dtype=torch.int16, device="cuda")
    g = B.gate(w.E, 8, balance_bias=torch.zeros(w.E))          # a bias in host memory
    for f, mode in ((B.moe_prefill_layer_gated, B.MODE_PREFILL), (B.moe_decode_layer_gated, B.MODE_DECODE)):
        with pytest.raises(ValueError):
            f(dw.dims, g, dw, x, torch.empty_like(x), T, ws=B.workspace(dw.dims, T, mode))
    logits, ok = torch.zeros((T, w.E), device="cuda"), B.gate(w.E, 8)
    out, ws = B.RouteBuffers(ok, T), B.gate_workspace(ok, T)
    with pytest.raises(ValueError):
        B.moe_route_gated(g, logits, T, out, ws)
    for bad in (ws[:1].expand(ws.numel()), ws.cpu(), ws.view(torch.int32)):
        with pytest.raises(ValueError):
            B.moe_route_gated(ok, logits, T, out, bad)
    with pytest.raises(ValueError):
        B.moe_route_gated(ok, logits.cpu(), T, out, ws)


def test_gated_layer_binding_wants_one_device():
    _, w, _ = synth.generate("tiny_t32", with_x=False)
    dw, T = B.DeviceWeights.from_logical(w), 2
    d, g, x = dw.dims, B.gate(w.E, 8), torch.zeros((T, w.H), dtype=torch.int16, device="cuda")
    for f, mode in ((B.moe_prefill_layer_gated, B.MODE_PREFILL), (B.moe_decode_layer_gated, B.MODE_DECODE)):
        ws = B.workspace(d, T, mode)
        for bad in (dict(y=x.cpu()), dict(ws=ws.cpu()), dict(logits_out=torch.zeros((T, w.E))),
                    dict(route_out=B.RouteBuffers(d, T, device="cpu"))):
            a = {**dict(y=torch.empty_like(x), ws=ws), **bad}
            with pytest.raises(ValueError, match=next(iter(bad))):
                f(d, g, dw, x, a.pop("y"), T, **a)
        with pytest.raises(ValueError, match="weights"):
            f(d, g, B.DeviceWeights.from_logical(w, device="cpu"), x, torch.empty_like(x), T, ws=ws)


def test_gated_layer_with_the_softmax_rule_is_the_layer():
    _, w, _ = synth.generate("tiny_t32", with_x=False)
    dw = B.DeviceWeights.from_logical(w)
    x = synth.make_x(np.random.default_rng(4), 40, w.H)
    d, g = dw.dims, B.gate()
    y = torch.empty((40, w.H), dtype=torch.int16, device="cuda")
    logits = torch.empty((40, w.E), device="cuda")
    ro = B.RouteBuffers(d, 40)
    B.moe_prefill_layer_gated(d, g, dw, torch.from_numpy(x).cuda(), y, 40, logits_out=logits, route_out=ro,
                              ws=B.workspace(d, 40, B.MODE_PREFILL))
    torch.cuda.synchronize()
    m = ro.to_numpy()
    check_layer(x, w, y.cpu().numpy().view(np.uint16), logits.cpu().numpy(), m["topk_idx"], m["topk_w"])


# ------------------------------------------------------------------ int4 projection with adapters

class _Matrix:
    def __init__(self, N, K, seed=0):
        g = torch.Generator().manual_seed(seed + N + K)
        self.N, self.K = N, K
        self.q = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
        self.s = (torch.rand((N, K // 64), generator=g) * 0.015 + 0.005).to(torch.bfloat16)
        self.b = (torch.rand((N, K // 64), generator=g) * 0.2 - 0.15).to(torch.bfloat16)
        bits = lambda t: t.view(torch.int16).numpy().view(np.uint16)[None]  # noqa: E731
        self.blob = torch.from_numpy(B.pack_int4_g64(self.q.numpy()[None], bits(self.s), bits(self.b))).cuda()


def _adapters(N, K, n, R, seed=0, full_rank=False):
    g = torch.Generator().manual_seed(seed + n + R)
    A = (torch.randn((n, R, K), generator=g) / K ** 0.5).to(torch.bfloat16)
    Bm = torch.randn((n, N, R), generator=g).to(torch.bfloat16)
    ranks = None if full_rank else torch.randint(0, R + 1, (n,), generator=g, dtype=torch.int32)
    scales = None if full_rank else torch.rand(n, generator=g) * 2 - 0.5
    return A, Bm, ranks, scales


def _dev(ts):
    return [None if t is None else t.cuda() for t in ts]


def _project(m, x, ad=None, of=None, gemm=B.GEMM_AUTO, pad=0, ws_fill=0xFF, stream=None):
    T = x.shape[0]
    xv, _ = _wide(x, pad, 0)
    yv, yf = _wide(torch.zeros((T, m.N), dtype=torch.bfloat16), pad, 1)
    a = B.Adapters(*_dev(ad)) if ad is not None else None
    ws = B.project_workspace(m.N, m.K, T, a)
    ws.fill_(ws_fill)
    B.moe_project(m.blob, m.N, m.K, xv, yv, T, a, None if of is None else of.cuda(), gemm, ws, stream)
    torch.cuda.synchronize()
    assert _behind(yf, T, m.N)
    return yv.cpu()


def _check_project(m, x, y, ad=None, of=None, wide=False):
    ref, tol = project_ref(x, m.q, m.s, m.b, *(ad or (None,) * 4), of=of, wide=wide)
    err = (y.double() - ref).abs()
    assert (err <= tol).all(), f"{(err / tol).max():.3f} of its bound"
    # the rounding of y, and of the weights where they are rounded, each at most 2^-8 relative
    rel = float(err.norm() / ref.norm())
    assert rel <= 2.0 ** -8 * (2 if wide else 1) + 1e-5, rel


def _x(T, K, seed=0):
    return torch.randn((T, K), generator=torch.Generator().manual_seed(seed + T)).to(torch.bfloat16)


def _runs(T, n, seed, none=0.2):
    """Tokens of requests: runs of random lengths with one adapter each, some with none."""
    rng = np.random.default_rng(seed)
    of = []
    while len(of) < T:
        a = -1 if rng.random() < none else int(rng.integers(n))
        of += [a] * int(rng.integers(1, max(2, T // 3)))
    return torch.tensor(of[:T], dtype=torch.int32)


GEMMS = [B.GEMM_AUTO, B.GEMM_EXACT, B.GEMM_WIDE]


@pytest.mark.parametrize("gemm", GEMMS)
@pytest.mark.parametrize("N,K", [(64, 128), (192, 256), (512, 2048), (2048, 512), (320, 4096), (64, 16384)])
def test_project_without_adapters(N, K, gemm):
    m = _Matrix(N, K)
    for T in (1, 2, 15, 16, 17, 33, 64, 100, 145, 300):
        x = _x(T, K)
        _check_project(m, x, _project(m, x, gemm=gemm), wide=gemm != B.GEMM_EXACT)


@pytest.mark.parametrize("gemm", GEMMS)
@pytest.mark.parametrize("R", [8, 16, 24, 64, 128])
@pytest.mark.parametrize("T", [1, 4, 16, 31, 64, 65, 150, 333])
def test_project_adapters(T, R, gemm):
    N, K, n = 192, 384, 7
    m = _Matrix(N, K)
    ad = _adapters(N, K, n, R)
    x = _x(T, K)
    rng = np.random.default_rng(T + R)
    each = torch.from_numpy(rng.integers(-1, n, T).astype(np.int32))     # every token its own choice
    for pad, of in ((0, each), (16, _runs(T, n, T + R)), (8, torch.full((T,), n - 1, dtype=torch.int32)),
                    (0, torch.full((T,), -1, dtype=torch.int32))):
        _check_project(m, x, _project(m, x, ad, of, gemm, pad), ad, of, wide=gemm != B.GEMM_EXACT)


@pytest.mark.parametrize("T,N,K,R,n", [(1, 4096, 2048, 16, 8), (32, 4096, 2048, 16, 32), (500, 2048, 2048, 32, 6),
                                       (1100, 1024, 2048, 16, 5), (64, 2048, 4096, 64, 64), (2, 512, 16384, 128, 2)])
def test_project_real_sizes(T, N, K, R, n):
    m = _Matrix(N, K)
    for full in (False, True):
        ad = _adapters(N, K, n, R, full_rank=full)
        x, of = _x(T, K), _runs(T, n, T)
        _check_project(m, x, _project(m, x, ad, of), ad, of, wide=True)


@pytest.mark.parametrize("N,K", [(64, 128), (192, 640), (4096, 2048), (6144, 2176), (12288, 512), (128, 16384)])
def test_project_few_tokens(N, K):
    # the projection's blocks form the adapters' first product themselves
    m, n = _Matrix(N, K), 3
    for T, R in ((1, 8), (1, 16), (1, 24), (1, 32), (1, 40), (2, 8), (2, 16), (3, 8), (4, 8), (5, 8), (1, 128)):
        ad = _adapters(N, K, n, R)
        x = _x(T, K)
        for of in ((torch.arange(T) % n).to(torch.int32), torch.full((T,), 1, dtype=torch.int32),
                   torch.full((T,), -1, dtype=torch.int32)):
            for gemm in (B.GEMM_AUTO, B.GEMM_EXACT):
                _check_project(m, x, _project(m, x, ad, of, gemm, pad=8), ad, of, wide=gemm != B.GEMM_EXACT)
    # a NaN adapter, what lies behind a rank, and a token of NaN
    A, Bm, _, scales = _adapters(N, K, 3, 8)
    ranks = torch.tensor([8, 5, 8], dtype=torch.int32)
    dirty = [A.clone(), Bm.clone(), ranks, scales]
    dirty[0][2, 3], dirty[0][1, 5:], dirty[1][1, :, 5:] = float("nan"), float("inf"), float("nan")
    x, of = _x(4, K), torch.tensor([1, 2, -1, 0], dtype=torch.int32)
    clean = _project(m, x, (A, Bm, ranks, scales), of)
    x[3] = float("nan")
    y = _project(m, x, dirty, of)
    assert torch.equal(y[[0, 2]], clean[[0, 2]])
    assert y[1].isnan().all() and y[3].isnan().all()


@pytest.mark.parametrize("T,R", [(1, 32), (2, 16), (4, 8)])
def test_project_one_launch_only_where_it_is_faster(T, R):
    # with T R = 32 rows every block read them all in two passes: 1.5 times the two launches' time, which more rows take
    N, K, n = 512, 16384, 4
    m, x = _Matrix(N, K), _x(T, K).cuda()
    y, of = torch.empty((T, N), dtype=torch.bfloat16, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    us = []
    for r in (R, R + 8):
        a = B.Adapters(*_dev(_adapters(N, K, n, r, full_rank=True)))
        ws = B.project_workspace(N, K, T, a)
        us.append(_graph_us(lambda: B.moe_project(m.blob, N, K, x, y, T, a, of, ws=ws)))
    assert us[0] < 1.25 * us[1], us


def test_project_adapter_names_out_of_range_mean_none():
    m, n = _Matrix(128, 256), 3
    ad = _adapters(128, 256, n, 8)
    for T in (5, 40):
        of = torch.tensor(([n, -7, 2 ** 31 - 1, -2 ** 31, 1] * 8)[:T], dtype=torch.int32)
        as_none = torch.where((of >= 0) & (of < n), of, torch.full_like(of, -1))
        assert torch.equal(_project(m, _x(T, 256), ad, of), _project(m, _x(T, 256), ad, as_none))


def test_project_ranks_out_of_range_are_limited():
    N, K, n, R = 128, 256, 5, 16
    m, (A, Bm, _, scales) = _Matrix(N, K), _adapters(N, K, n, R)
    ranks = torch.tensor([-1, 17, 2 ** 31 - 1, -2 ** 31, 9], dtype=torch.int32)
    for T in (1, 2, 40, 300):
        x, of = _x(T, K), torch.arange(T, dtype=torch.int32) % n
        if T == 1:
            of[0] = 2
        assert torch.equal(_project(m, x, (A, Bm, ranks, scales), of), _project(m, x, (A, Bm, ranks.clamp(0, R), scales), of))


@pytest.mark.parametrize("gemm", [B.GEMM_EXACT, B.GEMM_WIDE])
def test_project_widest(gemm):
    N, K, n, R = 65536, 128, 2, 8
    m, ad = _Matrix(N, K), _adapters(N, K, n, R)
    for T in (1, 3, 70):
        x, of = _x(T, K), torch.arange(T, dtype=torch.int32) % (n + 1) - 1
        _check_project(m, x, _project(m, x, ad, of, gemm), ad, of, wide=gemm == B.GEMM_WIDE)


@pytest.mark.parametrize("gemm", GEMMS)
def test_project_bad_values_reach_their_own_tokens_only(gemm):
    # an adapter of NaN and infinity beside others in the same tiles, garbage behind an adapter's rank,
    # and a token of NaN
    m, n, R = _Matrix(128, 256), 4, 16
    A, Bm, ranks, scales = _adapters(128, 256, n, R)
    ranks = torch.tensor([16, 5, 16, 0], dtype=torch.int32)
    dirty = [A.clone(), Bm.clone(), ranks, scales]
    dirty[0][2, 3], dirty[1][2, :, 1] = float("nan"), float("inf")
    dirty[0][1, 5:], dirty[1][1, :, 5:] = float("nan"), float("inf")
    dirty[0][3], dirty[1][3] = float("inf"), float("nan")
    for T in (8, 40, 200):
        x = _x(T, 256)
        of = torch.arange(T, dtype=torch.int32) % 5 - 1
        clean = _project(m, x, (A, Bm, ranks, scales), of, gemm)
        x[T // 2] = float("nan")
        y = _project(m, x, dirty, of, gemm)
        mine = (of != 2)
        mine[T // 2] = False
        assert torch.equal(y[mine], clean[mine])
        assert not y[T // 2].isfinite().any()
        assert y[of == 2].isnan().any()


@pytest.mark.parametrize("T", [1, 60, 300])
def test_project_many_adapters(T):
    # indices of more than eight bits, more distinct ones in a tile than a block's waves hold
    N, K, n, R = 128, 256, 700, 8
    m, ad, x = _Matrix(N, K), _adapters(N, K, n, R), _x(T, K)
    of = torch.from_numpy(np.random.default_rng(T).permutation(n)[:T].astype(np.int32))
    of[T // 2] = n - 1
    for gemm in GEMMS:
        _check_project(m, x, _project(m, x, ad, of, gemm), ad, of, wide=gemm != B.GEMM_EXACT)


@pytest.mark.parametrize("T", [3, 130, 260])
def test_widest_row_strides(T):
    # rows 2^20 elements apart: offsets inside a tile reach 2^29 bytes
    N, K, ld = 192, 256, 1 << 20
    m, ad, x = _Matrix(N, K), _adapters(N, K, 3, 16), _x(T, K)
    of = _runs(T, 3, T)
    a = B.Adapters(*_dev(ad))
    far = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")
    far[:, :K] = x.cuda()
    out = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")
    for gemm in GEMMS:
        B.moe_project(m.blob, N, K, far[:, :K], out[:, :N], T, a, of.cuda(), gemm, B.project_workspace(N, K, T, a))
        torch.cuda.synchronize()
        assert torch.equal(out[:, :N].cpu(), _project(m, x, ad, of, gemm))
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    B.moe_add_rmsnorm(B.norm(K), far[:, :K], w, T, y=out[:, :K])
    near = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    B.moe_add_rmsnorm(B.norm(K), x.cuda(), w, T, y=near)
    torch.cuda.synchronize()
    assert torch.equal(out[:, :K], near)


@pytest.mark.parametrize("T", [(1 << 18) + 300, 1 << 27])
def test_project_more_tokens_than_a_launch_takes(T):
    # a launch has fewer than 2^32 threads; the adapters' first product takes 32 a token
    N, K, R = 64, 128, 8
    m, ad = _Matrix(N, K), _adapters(N, K, 3, R, full_rank=True)
    a = B.Adapters(*_dev(ad))
    x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda").normal_()
    of = (torch.arange(T, dtype=torch.int32, device="cuda") % 5 - 1).clamp_(max=2)
    y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = B.project_workspace(N, K, T, a)
    ws.fill_(0xFF)
    B.moe_project(m.blob, N, K, x, y, T, a, of, B.GEMM_AUTO, ws)
    for t0 in (0, (1 << 18) - 40, T // 2 - 40, T - 80):
        at = slice(t0, t0 + 80)
        _check_project(m, x[at].cpu(), y[at].cpu(), ad, of[at].cpu(), wide=True)
    assert (y[T] == 7.0).all()
    del x, of, y, ws
    torch.cuda.empty_cache()


def test_project_results_do_not_depend_on_the_batch():
    # a token's result is the same bits alone in the call's tile and among others of the same call size
    m, n = _Matrix(256, 512), 5
    ad = _adapters(256, 512, n, 16)
    x = _x(48, 512)
    of = torch.arange(48, dtype=torch.int32) % n
    y = _project(m, x, ad, of)
    p = torch.randperm(48, generator=torch.Generator().manual_seed(1))
    assert torch.equal(_project(m, x[p], ad, of[p]), y[p])
    assert torch.equal(_project(m, x, ad, of), y)


# ------------------------------------------------------------------ streams, graphs, together

class _Block:
    """h = residual + x; xn = norm(h); p = projection(xn) with adapters; h2 = h + p; layer(norm(h2)), gated."""

    def __init__(self, T, seed=0):
        rng = np.random.default_rng(seed)
        _, self.w, _ = synth.generate("tiny_t32", with_x=False)
        self.dw = B.DeviceWeights.from_logical(self.w)
        H, self.T = self.w.H, T
        self.m = _Matrix(H, H)
        self.ad_host = _adapters(H, H, 4, 16)
        self.ad = B.Adapters(*_dev(self.ad_host))
        self.of = torch.from_numpy(rng.integers(-1, 4, T).astype(np.int32))
        self.bias = rng.uniform(-0.05, 0.05, 256).astype(np.float32)
        self.gate = B.gate(256, 8, score=B.SCORE_SIGMOID, n_groups=8, topk_groups=4, group_score=B.GROUP_TOP2, scale=2.5,
                           balance_bias=torch.from_numpy(self.bias).cuda())
        self.n = B.norm(H)
        self.wt = (torch.rand(H, generator=torch.Generator().manual_seed(seed)) + 0.5).to(torch.bfloat16)
        new = lambda: torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.x, self.res, self.h, self.xn, self.p, self.h2, self.xn2, self.y = (new() for _ in range(8))
        self.wd, self.ofd = self.wt.cuda(), self.of.cuda()
        self.logits = torch.zeros(T, 256, device="cuda")
        self.ro = B.RouteBuffers(self.dw.dims, T)
        self.ws_p = B.project_workspace(H, H, T, self.ad)
        self.ws_l = B.workspace(self.dw.dims, T, B.MODE_DECODE if T <= 4 else B.MODE_PREFILL)

    def run(self):
        T, H = self.T, self.w.H
        B.moe_add_rmsnorm(self.n, self.x, self.wd, T, residual=self.res, h_out=self.h, y=self.xn)
        B.moe_project(self.m.blob, H, H, self.xn, self.p, T, self.ad, self.ofd, ws=self.ws_p)
        B.moe_add_rmsnorm(self.n, self.p, self.wd, T, residual=self.h, h_out=self.h2, y=self.xn2)
        f = B.moe_decode_layer_gated if T <= 4 else B.moe_prefill_layer_gated
        f(self.dw.dims, self.gate, self.dw, self.xn2, self.y, T, logits_out=self.logits, route_out=self.ro, ws=self.ws_l)
        return [t.clone() for t in (self.h, self.xn, self.p, self.h2, self.xn2, self.logits, self.ro.topk_idx, self.y)]

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.x.copy_(torch.randn(self.x.shape, generator=g))
        self.res.copy_(torch.randn(self.x.shape, generator=g))


@pytest.mark.parametrize("T", [1, 4, 40])
def test_block_matches_64_bits(T):
    b = _Block(T)
    b.fill(T)
    h, xn, p, h2, xn2, logits, idx, y = [t.cpu() for t in b.run()]
    rel = norm_rel(b.w.H)
    want_h, v = norm_ref(b.x.cpu(), b.res.cpu(), b.wt, 1e-6, 0.0)
    assert torch.equal(h, want_h)
    assert ((xn.double() - v).abs() <= half_step(torch.bfloat16, v) * (1 + rel) + rel * v.abs()).all()
    _check_project(b.m, xn, p, b.ad_host, b.of, wide=True)
    want_h2, v = norm_ref(p, h, b.wt, 1e-6, 0.0)
    assert torch.equal(h2, want_h2)
    assert ((xn2.double() - v).abs() <= half_step(torch.bfloat16, v) * (1 + rel) + rel * v.abs()).all()
    want_idx, wsel = gate_ref(logits.numpy(), bias=b.bias, **GATE_DSV)
    assert np.array_equal(idx.numpy(), want_idx)
    ref = _layer_ref(xn2.view(torch.int16).numpy().view(np.uint16), b.w, want_idx, wsel)
    assert np.linalg.norm(y.double().numpy() - ref) / np.linalg.norm(ref) <= 5e-3


@pytest.mark.parametrize("T", [1, 40])
def test_block_in_a_graph(T):
    # replays with new inputs in between equal the eager results, and two graphs may share a workspace
    # as long as they run one after the other
    b = _Block(T)
    b.fill(0)
    b.run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = b.run()
        graphs.append((g, out))
    for seed in range(1, 5):
        b.fill(seed)
        want = b.run()
        torch.cuda.synchronize()
        for g, out in graphs:
            for t in out:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            for got, ref in zip(out, want):
                assert torch.equal(got, ref)


def test_block_on_two_streams():
    # two blocks with buffers of their own on two streams at once, several times
    bs = [_Block(40, 1), _Block(3, 2)]
    streams = [torch.cuda.Stream() for _ in bs]
    want = []
    for i, b in enumerate(bs):
        b.fill(10 + i)
        want.append(b.run())
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for b, s in zip(bs, streams):
            with torch.cuda.stream(s):
                got.append(b.run())
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, c in zip(g, w):
                assert torch.equal(a, c)


def test_empty_calls():
    n, g = B.norm(64), B.gate()
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    bf = dict(dtype=torch.bfloat16)
    B.moe_add_rmsnorm(n, z(0, 64, **bf), z(64, **bf), 0, y=z(0, 64, **bf))
    B.moe_route_gated(g, z(0, 256), 0, B.RouteBuffers(g, 0), B.gate_workspace(g, 0))
    m = _Matrix(64, 128)
    B.moe_project(m.blob, 64, 128, z(0, 128, **bf), z(0, 64, **bf), 0, ws=B.project_workspace(64, 128, 0))
    torch.cuda.synchronize()
