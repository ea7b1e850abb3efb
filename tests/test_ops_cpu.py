"""Host-side checks of the operators around the layer (no GPU needed): refusals of the C entry points
and of the binding, before anything would be launched, and the plain forms of perf/operators.py."""
import ctypes

import numpy as np
import pytest
import torch

from int4_grouped_gemm_router_amd import binding as B
from int4_grouped_gemm_router_amd import synth

FAKE = 0x10000  # never dereferenced: every call below returns before any launch
by = ctypes.byref


def _norm(n, x=FAKE, ldx=None, res=None, ldr=0, w=FAKE, h=None, ldh=0, y=FAKE, ldy=None, q=None, ldq=0, s=None, T=3):
    H = n.H if n is not None else 64
    return B.lib().moe_add_rmsnorm(by(n) if n is not None else None, x, H if ldx is None else ldx, res, ldr, w, h, ldh,
                                   y, H if ldy is None else ldy, q, ldq, s, T, None)


def test_norm_refusals():
    n = B.norm(64)
    assert _norm(n, T=0) == B.MOE_OK
    assert _norm(None) == B.MOE_EINVAL
    assert _norm(n, T=-1) == B.MOE_EINVAL
    assert _norm(n, x=None) == B.MOE_EINVAL
    assert _norm(n, w=None) == B.MOE_EINVAL
    assert _norm(n, y=None) == B.MOE_EINVAL                      # no output at all
    assert _norm(n, ldx=63) == B.MOE_EINVAL
    assert _norm(n, ldy=(1 << 20) + 1) == B.MOE_EINVAL
    assert _norm(n, x=FAKE + 1) == B.MOE_EINVAL                  # half an element
    assert _norm(n, w=FAKE + 1) == B.MOE_EINVAL
    assert _norm(n, q=FAKE, ldq=64, s=FAKE) == B.MOE_EINVAL      # 8-bit buffers without an 8-bit output
    n8 = B.norm(64, out8=B.OUT8_INT8, group=32)
    assert _norm(n8) == B.MOE_EINVAL                             # and the reverse
    assert _norm(n8, q=FAKE, ldq=64) == B.MOE_EINVAL             # q without scales
    assert _norm(n8, q=FAKE, ldq=63, s=FAKE) == B.MOE_EINVAL
    assert _norm(n8, q=FAKE, ldq=64, s=FAKE + 2) == B.MOE_EINVAL
    # in place only with the row stride of what is replaced
    assert _norm(n, ldx=128, y=FAKE, ldy=64) == B.MOE_EINVAL
    assert _norm(n, res=FAKE + 0x4000, ldr=64, h=FAKE + 0x4000, ldh=72) == B.MOE_EINVAL
    for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(weight_offset=float("inf")), dict(out8=3)):
        assert _norm(B.norm(64, **bad)) == B.MOE_EINVAL, bad
    for bad in (dict(H=0), dict(H=16385), dict(H=96, group=64), dict(H=96, group=48), dict(H=64, group=-32)):
        assert _norm(B.norm(**bad)) == B.MOE_EUNSUPPORTED, bad
    assert _norm(B.MoeNorm(64, 3, 3, 0, 0, 1e-6, 0.0)) == B.MOE_EINVAL
    assert _norm(B.MoeNorm(64, B.BF16, B.F16, 0, 0, 1e-6, 0.0)) == B.MOE_EINVAL
    with pytest.raises(ValueError):
        B.norm(64, dtype=torch.float64)


def test_norm_binding_checks_tensors():
    n = B.norm(64)
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    y = torch.empty_like(x)
    for kw in (dict(x=x.float(), y=y), dict(x=x[:, :32], y=y), dict(x=x, y=y[:2]), dict(x=x.t().contiguous().t(), y=y),
               dict(x=x, y=y, residual=x.half())):
        with pytest.raises(ValueError):
            B.moe_add_rmsnorm(n, kw.pop("x"), w, 4, **kw)
    with pytest.raises(ValueError):
        B.moe_add_rmsnorm(n, x, w[:32], 4, y=y)
    with pytest.raises(ValueError):      # the checks pass; there is no CPU path
        B.moe_add_rmsnorm(n, x, w, 4, y=y)


GATES_BAD_VALUE = [dict(score=2), dict(score=-1), dict(group_score=2), dict(renorm=2), dict(scale=float("nan")),
                   dict(scale=float("inf"))]
GATES_UNSUPPORTED = [dict(E=0, top_k=1), dict(E=257), dict(top_k=0), dict(top_k=17), dict(E=4, top_k=5), dict(block_m=64),
                     dict(n_groups=0), dict(n_groups=3), dict(E=256, n_groups=128, topk_groups=128),
                     dict(n_groups=8, topk_groups=0), dict(n_groups=8, topk_groups=9),
                     dict(E=64, n_groups=16, topk_groups=1, top_k=8)]


def _gate(**kw):
    a = dict(E=256, top_k=8, block_m=32, score=0, n_groups=1, topk_groups=1, group_score=0, renorm=1, scale=1.0)
    a.update(kw)
    return B.MoeGate(*[a[f] for f, _ in B.MoeGate._fields_[:-1]], None)


def test_gate_refusals():
    L = B.lib()
    g = _gate()
    ro = B.MoeRouteOut(*([FAKE] * 8))
    n = ctypes.c_size_t(0)
    assert L.moe_gate_workspace_bytes(by(g), 64, by(n)) == B.MOE_OK and n.value > 0
    assert L.moe_gate_max_blocks(by(g), 512) == 512 * 8 // 32 + 256
    for bad in GATES_BAD_VALUE:
        assert L.moe_gate_workspace_bytes(by(_gate(**bad)), 64, by(n)) == B.MOE_EINVAL, bad
        assert L.moe_route_gated(by(_gate(**bad)), FAKE, 4, by(ro), FAKE, 1 << 30, None) == B.MOE_EINVAL, bad
    for bad in GATES_UNSUPPORTED:
        assert L.moe_gate_workspace_bytes(by(_gate(**bad)), 64, by(n)) == B.MOE_EUNSUPPORTED, bad
        assert L.moe_route_gated(by(_gate(**bad)), FAKE, 4, by(ro), FAKE, 1 << 30, None) == B.MOE_EUNSUPPORTED, bad
    g.balance_bias = FAKE + 2
    assert L.moe_route_gated(by(g), FAKE, 4, by(ro), FAKE, 1 << 30, None) == B.MOE_EINVAL
    g.balance_bias = None
    assert L.moe_route_gated(None, FAKE, 4, by(ro), FAKE, 1 << 30, None) == B.MOE_EINVAL
    assert L.moe_route_gated(by(g), FAKE, 0, by(ro), None, 0, None) == B.MOE_OK
    assert L.moe_route_gated(by(g), FAKE, -1, by(ro), FAKE, 1 << 30, None) == B.MOE_EINVAL
    assert L.moe_route_gated(by(g), None, 4, by(ro), FAKE, 1 << 30, None) == B.MOE_EINVAL
    assert L.moe_route_gated(by(g), FAKE, 4, None, FAKE, 1 << 30, None) == B.MOE_EINVAL
    assert L.moe_route_gated(by(g), FAKE, 4, by(ro), FAKE, 0, None) == B.MOE_EWORKSPACE
    assert L.moe_route_gated(by(g), FAKE, 4, by(ro), FAKE + 8, 1 << 30, None) == B.MOE_EINVAL
    assert L.moe_route_gated(by(g), FAKE, 1 << 27, by(ro), FAKE, 1 << 40, None) == B.MOE_EUNSUPPORTED


def test_gate_refuses_more_tokens_than_a_launch_takes():
    # sixteen threads a token, fewer than 2^32 a launch
    L, n, most = B.lib(), ctypes.c_size_t(0), (1 << 28) - 64
    ro = B.MoeRouteOut(*([FAKE] * 8))
    for k in (1, 2, 3):
        g = _gate(E=4, top_k=k)
        assert L.moe_gate_workspace_bytes(by(g), most, by(n)) == B.MOE_OK
        assert L.moe_gate_workspace_bytes(by(g), most + 1, by(n)) == B.MOE_EUNSUPPORTED
        assert L.moe_route_gated(by(g), FAKE, most + 1, by(ro), FAKE, 1 << 40, None) == B.MOE_EUNSUPPORTED
        assert L.moe_route_gated(by(g), FAKE, most, by(ro), FAKE, 0, None) == B.MOE_EWORKSPACE


def test_gate_workspace_serves_fewer_tokens():
    n, most = ctypes.c_size_t(0), 0
    for T in sorted([*range(0, 20000, 7), 64, 4096, 4097, 8192, 8193, 16384, 16385, 32769, 1 << 20]):
        assert B.lib().moe_gate_workspace_bytes(by(_gate()), T, by(n)) == B.MOE_OK
        assert n.value >= most, T
        most = n.value


def test_gated_layer_refusals():
    L = B.lib()
    d, w = B.dims(2048, 512), B.MoeLayerWeights(*([FAKE] * 7))
    ws = B.moe_workspace_bytes(d, 64, B.MODE_PREFILL)

    def prefill(dd, g, T=64, n=ws):
        return L.moe_prefill_layer_gated(by(dd), by(g) if g is not None else None, by(w), FAKE, FAKE, T, 0, None, None,
                                         FAKE, n, None)

    def decode(dd, g, T=1):
        return L.moe_decode_layer_gated(by(dd), by(g) if g is not None else None, by(w), FAKE, FAKE, T, None, None, FAKE,
                                        0, None)

    for f in (prefill, decode):
        assert f(d, None) == B.MOE_EINVAL
        assert f(d, _gate(score=7)) == B.MOE_EINVAL
        assert f(d, _gate(E=128)) == B.MOE_EINVAL                # not the layer's experts
        assert f(d, _gate(top_k=4)) == B.MOE_EINVAL
        assert f(d, _gate(block_m=16)) == B.MOE_EINVAL
        assert f(B.dims(2048, 512, top_k=4), _gate(top_k=4)) == B.MOE_EUNSUPPORTED
        assert f(d, _gate(), T=0) == B.MOE_OK
        assert f(d, _gate(), T=-1) == B.MOE_EINVAL
    assert prefill(d, _gate(), n=ws - 1) == B.MOE_EWORKSPACE
    assert decode(d, _gate()) == B.MOE_EWORKSPACE
    assert decode(d, _gate(), T=5) == B.MOE_EUNSUPPORTED


@pytest.mark.parametrize("f,mode", [(B.moe_prefill_layer_gated, B.MODE_PREFILL), (B.moe_decode_layer_gated, B.MODE_DECODE)])
def test_gated_layer_binding_checks_tensors(f, mode):
    _, w, _ = synth.generate("tiny_t32", with_x=False)
    dw, T = B.DeviceWeights.from_logical(w, device="cpu"), 3
    d, g = dw.dims, B.gate(w.E, 8)
    x = torch.zeros((T, w.H), dtype=torch.bfloat16)
    ok = dict(x=x, y=torch.empty_like(x), logits_out=torch.empty((T, w.E)), route_out=B.RouteBuffers(d, T, device="cpu"),
              ws=B.workspace(d, T, mode, device="cpu"))

    def call(**kw):
        a = {**ok, **kw}
        f(d, g, dw, a.pop("x"), a.pop("y"), T, **a)

    for kw in (dict(x=x.float()), dict(x=x.half()), dict(x=x[:2]), dict(x=torch.zeros((T, 2 * w.H), dtype=x.dtype)[:, ::2]),
               dict(y=x[:2].clone()), dict(y=x.float()), dict(y=torch.zeros((w.H, T), dtype=x.dtype).t()),
               dict(logits_out=torch.empty((T - 1, w.E))), dict(logits_out=torch.empty((T, w.E), dtype=torch.float64)),
               dict(route_out=B.RouteBuffers(d, T - 1, device="cpu")), dict(ws=ok["ws"].view(torch.int32)),
               dict(ws=ok["ws"][::2])):
        with pytest.raises(ValueError, match=next(iter(kw))):
            call(**kw)
    for dtype in (torch.bfloat16, torch.int16, torch.uint16):      # the checks pass; there is no CPU path
        with pytest.raises(ValueError, match="on a GPU"):
            call(x=x.view(dtype), y=x.clone().view(dtype))


def test_gated_prefill_binding_wants_the_last_chunks_buffers():
    _, w, _ = synth.generate("tiny_t32", with_x=False)
    dw, T, chunk = B.DeviceWeights.from_logical(w, device="cpu"), 50, 16
    x, g = torch.zeros((T, w.H), dtype=torch.bfloat16), B.gate(w.E, 8)
    for tokens, match in ((2, "on a GPU"), (1, "route_out")):      # 50 = 3 * 16 + 2
        with pytest.raises(ValueError, match=match):
            B.moe_prefill_layer_gated(dw.dims, g, dw, x, torch.empty_like(x), T, chunk,
                                      route_out=B.RouteBuffers(dw.dims, tokens, device="cpu"),
                                      ws=B.workspace(dw.dims, chunk, B.MODE_PREFILL, device="cpu"))


def _project(blob=FAKE, N=128, K=256, x=FAKE, ldx=256, y=FAKE, ldy=128, T=4, ad=None, of=None, gemm=0, ws=FAKE, n=1 << 30):
    return B.lib().moe_project(blob, N, K, x, ldx, y, ldy, T, by(ad) if ad is not None else None, of, gemm, ws, n, None)


def test_project_refusals():
    ad = lambda **kw: B.MoeAdapters(**{**dict(n=2, R=16, A=FAKE, B=FAKE, ranks=None, scales=None), **kw})  # noqa: E731
    assert _project(T=0) == B.MOE_OK
    assert _project(T=-1) == B.MOE_EINVAL
    for kw in (dict(blob=None), dict(x=None), dict(y=None), dict(x=FAKE + 8), dict(y=FAKE + 2), dict(blob=FAKE + 4),
               dict(ldx=255), dict(ldx=260), dict(ldy=120), dict(ldy=132), dict(ldx=(1 << 20) + 8), dict(ws=FAKE + 8),
               dict(gemm=3), dict(gemm=-1), dict(of=FAKE), dict(ad=ad())):
        assert _project(**kw) == B.MOE_EINVAL, kw
    for kw in (dict(N=96), dict(N=0), dict(N=65600), dict(K=192), dict(K=0), dict(K=16512, ldx=16512)):
        assert _project(**kw) == B.MOE_EUNSUPPORTED, kw
    for kw in (dict(n=0), dict(A=None), dict(B=None), dict(A=FAKE + 8), dict(B=FAKE + 2), dict(ranks=FAKE + 1),
               dict(scales=FAKE + 2)):
        assert _project(ad=ad(**kw), of=FAKE) == B.MOE_EINVAL, kw
    for R in (0, 4, 12, 136, -8):
        assert _project(ad=ad(R=R), of=FAKE) == B.MOE_EUNSUPPORTED, R
    assert _project(ad=ad(), of=FAKE + 2) == B.MOE_EINVAL
    n = ctypes.c_size_t(0)
    L = B.lib()
    assert L.moe_project_workspace_bytes(128, 256, 16, 4, by(n)) == B.MOE_OK and n.value > 0
    assert _project(ad=ad(), of=FAKE, n=n.value - 1) == B.MOE_EWORKSPACE
    assert _project(ad=ad(), of=FAKE, ws=None, n=0) == B.MOE_EINVAL
    assert L.moe_project_workspace_bytes(128, 256, 12, 4, by(n)) == B.MOE_EUNSUPPORTED
    assert L.moe_project_workspace_bytes(100, 256, 8, 4, by(n)) == B.MOE_EUNSUPPORTED
    assert L.moe_project_workspace_bytes(128, 256, 8, -1, by(n)) == B.MOE_EINVAL
    assert L.moe_project_workspace_bytes(128, 256, 8, 4, None) == B.MOE_EINVAL
    assert L.moe_project_workspace_bytes(128, 256, 8, (1 << 30) + 1, by(n)) == B.MOE_EUNSUPPORTED
    assert _project(T=(1 << 30) + 1) == B.MOE_EUNSUPPORTED
    assert _project(T=0x7FFFFFFF) == B.MOE_EUNSUPPORTED


def test_unknown_types_are_refused_by_the_binding():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    for n in (B.MoeNorm(64, 3, 3, 0, 0, 1e-6, 0.0), B.MoeNorm(64, -1, 0, 0, 0, 1e-6, 0.0), B.norm(64, out8=7)):
        with pytest.raises(ValueError):
            B.moe_add_rmsnorm(n, x, w, 2, y=torch.empty_like(x), q=torch.zeros(2, 64, dtype=torch.int8),
                              scales=torch.zeros(2))


def test_project_binding_checks_tensors():
    N, K, T = 64, 128, 4
    blob = torch.from_numpy(B.pack_int4_g64(np.zeros((1, N, K), np.uint8), np.zeros((1, N, 2), np.uint16),
                                            np.zeros((1, N, 2), np.uint16)))
    bf = dict(dtype=torch.bfloat16)
    x, y = torch.zeros(T, K, **bf), torch.zeros(T, N, **bf)
    A, Bm = torch.zeros(3, 8, K, **bf), torch.zeros(3, N, 8, **bf)
    with pytest.raises(ValueError):
        B.Adapters(A, Bm.transpose(1, 2))
    with pytest.raises(ValueError):
        B.Adapters(A.float(), Bm.float())
    with pytest.raises(ValueError):
        B.Adapters(A, Bm, ranks=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        B.Adapters(A, Bm, scales=torch.zeros(3, dtype=torch.float64))
    ad = B.Adapters(A, Bm)
    of = torch.zeros(T, dtype=torch.int32)
    for args, kw in (((blob[:-1], N, K, x, y, T), {}), ((blob, N, K, x[:2], y, T), {}), ((blob, N, K, x, y[:, :32], T), {}),
                     ((blob, N, K, x.float(), y, T), {}), ((blob, N, K, x, y, T), dict(adapters=ad, adapter_of=of.long())),
                     ((blob, N, K, x, y, T), dict(adapters=ad, adapter_of=of[:2])),
                     ((blob, N, K, x, y, T), dict(adapters=B.Adapters(torch.zeros(3, 8, 256, **bf), Bm), adapter_of=of))):
        with pytest.raises(ValueError):
            B.moe_project(*args, **kw)
