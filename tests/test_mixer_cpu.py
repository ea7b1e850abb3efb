"""Host-side checks of the operators of a block's mixer half (no GPU needed): refusals of the C entry points and of
the binding, before anything would be launched, and the frequencies of rotary positions."""
import ctypes
import math

import numpy as np
import pytest
import torch

from int4_grouped_gemm_router_amd import binding as B

FAKE = 0x10000  # never dereferenced: every call below returns before any launch
by = ctypes.byref


# ------------------------------------------------------------------ int8 projection

def _int8(w=FAKE, ws=FAKE, bias=None, N=64, K=128, x=FAKE, ldx=None, xs=FAKE, y=FAKE, ldy=None, dtype=B.BF16, T=3, work=FAKE,
          n=1 << 40):
    return B.lib().moe_project_int8(w, ws, bias, N, K, x, K if ldx is None else ldx, xs, y, N if ldy is None else ldy, dtype, T,
                                    work, n, None)


def test_int8_refusals():
    assert _int8(T=0, w=None, x=None, y=None) == B.MOE_OK
    for bad in (dict(T=-1), dict(dtype=3), dict(dtype=-1), dict(w=None), dict(ws=None), dict(x=None), dict(xs=None), dict(y=None),
                dict(w=FAKE + 8), dict(x=FAKE + 8), dict(ws=FAKE + 2), dict(xs=FAKE + 2), dict(bias=FAKE + 1), dict(y=FAKE + 1),
                dict(dtype=B.F32, y=FAKE + 2), dict(ldx=127), dict(ldx=136), dict(ldx=112), dict(ldx=(1 << 20) + 16), dict(ldy=63),
                dict(ldy=(1 << 20) + 1), dict(work=FAKE + 8)):
        assert _int8(**bad) == B.MOE_EINVAL, bad
    for bad in (dict(N=0), dict(N=(1 << 18) + 1), dict(K=0), dict(K=32), dict(K=96), dict(K=65600), dict(T=(1 << 30) + 1)):
        assert _int8(**bad) == B.MOE_EUNSUPPORTED, bad
    n = ctypes.c_size_t(7)
    f = B.lib().moe_project_int8_workspace_bytes
    assert f(64, 128, 3, None) == B.MOE_EINVAL and f(64, 128, -1, by(n)) == B.MOE_EINVAL and f(64, 96, 3, by(n)) == B.MOE_EUNSUPPORTED
    assert f(64, 128, 0, by(n)) == B.MOE_OK


def test_int8_workspace_is_demanded():
    n = ctypes.c_size_t(0)
    for N, K, T in ((12288, 2048, 1), (256, 65536, 4), (64, 64, 1), (4096, 4096, 300)):
        assert B.lib().moe_project_int8_workspace_bytes(N, K, T, by(n)) == B.MOE_OK
        if n.value:
            assert _int8(N=N, K=K, T=T, n=n.value - 1) == B.MOE_EWORKSPACE
            assert _int8(N=N, K=K, T=T, work=None, n=n.value) == B.MOE_EINVAL


def test_int8_binding_checks_tensors():
    w, ws, x, xs = torch.zeros(32, 64, dtype=torch.int8), torch.zeros(32), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    y = torch.zeros(4, 32)
    for kw in (dict(w=w.float()), dict(w=w[0]), dict(ws=ws[:31]), dict(x=x[:, :32]), dict(x=x.float()), dict(xs=xs[:3]),
               dict(y=y.double()), dict(y=y[:3]), dict(y=y[:, :31]), dict(bias=ws[:5]), dict(bias=ws.double())):
        a = dict(w=w, ws=ws, x=x, xs=xs, y=y, bias=None)
        a.update(kw)
        with pytest.raises(ValueError):
            B.moe_project_int8(a["w"], a["ws"], a["x"], a["xs"], a["y"], 4, bias=a["bias"])
    with pytest.raises(ValueError):      # the checks pass; there is no CPU path
        B.moe_project_int8(w, ws, x, xs, y, 4)


# ------------------------------------------------------------------ rotary positions

def test_rope_radians_follow_the_formulas():
    rot, base = 64, 1e6
    plain = base ** (-np.arange(0, rot, 2) / rot)
    r, m = B.rope_radians(rot, base)
    assert np.allclose(r, plain, rtol=1e-14, atol=0) and m == 1.0
    r, m = B.rope_radians(rot, base, B.ROPE_LINEAR, 4.0)
    assert np.allclose(r, plain / 4, rtol=1e-14, atol=0) and m == 1.0
    r, m = B.rope_radians(rot, base, B.ROPE_NTK, 4.0)
    assert np.allclose(r, (base * 4.0 ** (64 / 62)) ** (-np.arange(0, rot, 2) / rot), rtol=1e-13, atol=0) and m == 1.0
    assert math.isclose(r[-1], plain[-1] / 4, rel_tol=1e-12)          # the slowest pair is stretched by the factor
    r, m = B.rope_radians(rot, base, B.ROPE_YARN, 4.0, 4096)
    turns = 4096 * plain / (2 * math.pi)
    assert (r[turns >= 32] == plain[turns >= 32]).all() and np.allclose(r[turns <= 1], plain[turns <= 1] / 4, rtol=1e-14)
    assert (np.diff(r) < 0).all() and math.isclose(m, 0.1 * math.log(4) + 1, rel_tol=1e-7)
    one, m1 = B.rope_radians(rot, base, B.ROPE_YARN, 1.0, 4096)
    assert np.allclose(one, plain, rtol=1e-14) and m1 == 1.0


def test_rope_turns_are_exact_fractions():
    rad = np.array([0.0, math.pi, math.pi / 2, -math.pi / 2, 2 * math.pi * 7, 1.0])
    out = np.empty(6, np.uint64)
    assert B.lib().moe_rope_turns(rad.ctypes.data, 6, out.ctypes.data) == B.MOE_OK
    want = [0, 1 << 63, 1 << 62, 3 << 62, 0, int(2 ** 64 / (2 * math.pi))]
    for o, w in zip(out.tolist(), want):
        d = (o - w) % (1 << 64)
        assert min(d, (1 << 64) - d) <= 1 << 15          # float64's own step of pi
    rad[2] = math.inf
    assert B.lib().moe_rope_turns(rad.ctypes.data, 6, out.ctypes.data) == B.MOE_EINVAL
    assert B.lib().moe_rope_turns(None, 6, out.ctypes.data) == B.MOE_EINVAL
    assert B.lib().moe_rope_turns(rad.ctypes.data, -1, out.ctypes.data) == B.MOE_EINVAL


def test_rope_scaling_refusals():
    for bad in (dict(base=0.0), dict(base=-1.0), dict(base=math.inf), dict(scaling=4), dict(scaling=-1),
                dict(scaling=B.ROPE_LINEAR, factor=0.5), dict(scaling=B.ROPE_NTK, factor=math.nan),
                dict(scaling=B.ROPE_YARN, factor=2.0), dict(scaling=B.ROPE_YARN, factor=2.0, context=100, slow=3.0, fast=3.0)):
        with pytest.raises(B.MoeError) as e:
            B.rope_radians(64, **bad)
        assert e.value.code == B.MOE_EINVAL, bad
    for rot, kind in ((0, 0), (3, 0), (1026, 0), (2, B.ROPE_NTK), (-2, 0)):
        with pytest.raises(B.MoeError) as e:
            B.rope_radians(rot, scaling=kind, factor=2.0)
        assert e.value.code == B.MOE_EUNSUPPORTED, rot
    with pytest.raises(ValueError):
        B.rope(64, radians=np.ones(31), device="cpu")


def _rotary(**kw):
    a = dict(head_dim=64, rot_dim=32, dtype=B.BF16, interleaved=0, inverse=0, magnitude=1.0, turns=FAKE)
    a.update(kw)
    return B.MoeRotary(*[a[f] for f, _ in B.MoeRotary._fields_])


def _rope(r=None, q=FAKE, ldq=256, qo=FAKE, ldqo=256, hq=4, k=None, ldk=0, ko=None, ldko=0, hk=0, p=FAKE, T=3):
    return B.lib().moe_rope(by(r or _rotary()), q, ldq, qo, ldqo, hq, k, ldk, ko, ldko, hk, p, T, None)


def test_rope_refusals():
    assert _rope(T=0, q=None) == B.MOE_OK
    assert B.lib().moe_rope(None, FAKE, 256, FAKE, 256, 4, None, 0, None, 0, 0, FAKE, 3, None) == B.MOE_EINVAL
    for bad in (dict(T=-1), dict(q=None), dict(qo=None), dict(p=None), dict(p=FAKE + 2), dict(q=FAKE + 1), dict(ldq=255), dict(ldqo=128),
                dict(ldq=(1 << 20) + 1, qo=FAKE * 2), dict(ldqo=264), dict(k=FAKE, hk=2, ldk=128), dict(ko=FAKE),
                dict(k=FAKE, ko=FAKE * 2, hk=2, ldk=127, ldko=128), dict(k=FAKE, ko=FAKE, hk=2, ldk=128, ldko=136)):
        assert _rope(**bad) == B.MOE_EINVAL, bad
    for bad in (dict(hq=0), dict(hq=1025, ldq=1 << 17, ldqo=1 << 17), dict(k=FAKE, ko=FAKE, hk=0), dict(T=(1 << 30) + 1)):
        assert _rope(**bad) == B.MOE_EUNSUPPORTED, bad
    for bad in (dict(dtype=3), dict(interleaved=2), dict(inverse=-1), dict(magnitude=math.nan), dict(turns=None), dict(turns=FAKE + 4)):
        assert _rope(_rotary(**bad)) == B.MOE_EINVAL, bad
    for bad in (dict(head_dim=1025), dict(rot_dim=66), dict(rot_dim=31), dict(rot_dim=0), dict(head_dim=1, rot_dim=1)):
        assert _rope(_rotary(**bad)) == B.MOE_EUNSUPPORTED, bad


def test_rope_binding_checks_tensors():
    r = B.rope(64, 32, device="cpu")
    q, p = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32)
    for kw in (dict(q=q.float()), dict(q=q[:4]), dict(p=p.long()), dict(p=p[:4]), dict(q=q[:, :, :32]), dict(q_out=q[:, :3].contiguous()),
               dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(k_out=q), dict(k=q, k_out=q[:, :2])):
        a = dict(q=q, p=p)
        a.update(kw)
        with pytest.raises(ValueError):
            B.moe_rope(r, a.pop("p"), 5, a.pop("q"), **a)
    with pytest.raises(ValueError):      # the checks pass; there is no CPU path
        B.moe_rope(r, p, 5, q)


# ------------------------------------------------------------------ linear attention

def _plan(**kw):
    a = dict(qk_heads=2, v_heads=4, qk_dim=64, v_dim=32, scale=1.0)
    a.update(kw)
    return B.MoeLinear(*[a[f] for f, _ in B.MoeLinear._fields_])


def _linear(l=None, q=FAKE, ldq=128, k=FAKE, ldk=128, v=FAKE, ldv=128, g=FAKE, ldg=4, cu=FAKE, n=2, si=FAKE, sli=None, ni=2, so=FAKE,
            slo=None, no=2, o=FAKE, ldo=128, T=9, ws=FAKE, wn=1 << 50, step=False):
    L = B.lib()
    head = (by(l or _plan()), q, ldq, k, ldk, v, ldv, g, ldg)
    states = (si, sli, ni, so, slo, no, o, ldo, T)
    if step:
        return L.moe_linear_attention_step(*head, *states, None)
    return L.moe_linear_attention(*head, cu, n, *states, ws, wn, None)


LINEAR_BAD = [dict(T=-1), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(g=None), dict(q=FAKE + 8), dict(o=FAKE + 2),
              dict(g=FAKE + 2), dict(ldq=120), dict(ldk=132), dict(ldv=(1 << 20) + 8), dict(ldo=64), dict(ldg=3), dict(ldg=-4),
              dict(ni=0), dict(no=0), dict(si=FAKE + 4), dict(so=FAKE + 8), dict(si=None, sli=FAKE), dict(so=None, slo=FAKE),
              dict(sli=FAKE + 2), dict(slo=FAKE + 1)]


def test_linear_refusals():
    for step in (False, True):
        for bad in LINEAR_BAD:
            assert _linear(step=step, **bad) == B.MOE_EINVAL, bad
        for bad in (dict(qk_heads=0), dict(qk_heads=3), dict(v_heads=0), dict(v_heads=1026), dict(qk_dim=4), dict(qk_dim=60),
                    dict(qk_dim=264), dict(v_dim=0), dict(v_dim=264)):
            assert _linear(_plan(**bad), step=step) == B.MOE_EUNSUPPORTED, bad
        assert _linear(_plan(scale=math.nan), step=step) == B.MOE_EINVAL
    assert _linear(n=0, q=None, cu=None) == B.MOE_OK
    assert _linear(T=0, q=None, step=True) == B.MOE_OK
    assert _linear(n=-1) == B.MOE_EINVAL
    assert _linear(cu=None) == B.MOE_EINVAL
    assert _linear(cu=FAKE + 2) == B.MOE_EINVAL
    assert _linear(n=65537) == B.MOE_EUNSUPPORTED
    assert _linear(T=(1 << 30) + 1) == B.MOE_EUNSUPPORTED
    assert _linear(T=65537, step=True) == B.MOE_EUNSUPPORTED
    n = ctypes.c_size_t(0)
    f = B.lib().moe_linear_workspace_bytes
    assert f(None, 1, 1, by(n)) == B.MOE_EINVAL and f(by(_plan()), -1, 1, by(n)) == B.MOE_EINVAL
    assert f(by(_plan()), 1, 1, None) == B.MOE_EINVAL and f(by(_plan(qk_dim=12)), 1, 1, by(n)) == B.MOE_EUNSUPPORTED


def test_linear_workspace_is_demanded_and_serves_fewer():
    n = ctypes.c_size_t(0)
    f = B.lib().moe_linear_workspace_bytes
    l = _plan(qk_heads=16, v_heads=32, qk_dim=128, v_dim=128)
    wide = dict(ldq=2048, ldk=2048, ldv=4096, ldo=4096, ldg=32)
    for seqs in (1, 4, 64):
        most = 0
        for T in sorted([*range(0, 3000, 37), 4096, 8191, 8192, 16384, 65536, 1 << 20]):
            assert f(by(l), seqs, T, by(n)) == B.MOE_OK
            assert n.value >= most, (seqs, T)
            most = n.value
        if most:
            assert _linear(l, n=seqs, T=1 << 20, wn=most - 1, **wide) == B.MOE_EWORKSPACE
            assert _linear(l, n=seqs, T=1 << 20, wn=most, ws=None, **wide) == B.MOE_EINVAL
            assert _linear(l, n=seqs, T=1 << 20, wn=most, ws=FAKE + 8, **wide) == B.MOE_EINVAL
    for T in (100, 5000, 16384):
        most = 0
        for seqs in (1, 2, 3, 5, 8, 17, 64, 300, 5000):
            assert f(by(l), seqs, T, by(n)) == B.MOE_OK
            assert n.value >= most, (seqs, T)
            most = n.value


def test_linear_binding_checks_tensors():
    l = B.linear_attention(2, 4, 64, 32)
    T = 6
    a = dict(q=torch.zeros(T, 2, 64), k=torch.zeros(T, 2, 64), v=torch.zeros(T, 4, 32), o=torch.zeros(T, 4, 32))
    a = {n: t.bfloat16() for n, t in a.items()}
    a.update(g=torch.zeros(T, 4), cu=torch.tensor([0, 6], dtype=torch.int32), state_in=None, slots_in=None, state_out=None,
             slots_out=None)
    S, slots = torch.zeros(2, 4, 64, 32), torch.zeros(1, dtype=torch.int32)

    def call(**kw):
        c = dict(a)
        c.update(kw)
        B.moe_linear_attention(l, c["q"], c["k"], c["v"], c["g"], c["o"], c["cu"], T,
                               **{n: c[n] for n in ("state_in", "slots_in", "state_out", "slots_out")})
    for bad in (dict(q=a["q"].float()), dict(q=a["q"][:5]), dict(k=a["k"][:, :1]), dict(v=a["q"]), dict(o=a["o"][:, :, :16]),
                dict(g=a["g"].double()), dict(g=a["g"][:5]), dict(g=a["g"][0, :3]), dict(g=torch.zeros(5)), dict(cu=a["cu"].long()),
                dict(cu=a["cu"][:0]), dict(state_in=S.double()), dict(state_in=S[:, :, :, :16]), dict(state_in=S[0]), dict(slots_in=slots),
                dict(state_in=S, slots_in=slots[:0]), dict(state_out=S, slots_out=slots.long()), dict(slots_out=slots), dict()):
        with pytest.raises(ValueError):  # (the last: every check passes; there is no CPU path)
            call(**bad)


# ------------------------------------------------------------------ the norm after a block

def _gated(n, x=FAKE, ldx=None, w=None, gate=None, ldg=0, c=None, r=None, ldr=0, nw=None, h=FAKE, ldh=None, y=None, ldy=0, q=None, ldq=0,
           s=None, T=3):
    H = n.H if n is not None else 64
    return B.lib().moe_gated_norm(by(n) if n is not None else None, x, H if ldx is None else ldx, w, gate, ldg, c, r, ldr, nw, h,
                                  H if ldh is None else ldh, y, ldy, q, ldq, s, T, None)


def test_gated_refusals():
    n = B.gated_norm(64)
    assert _gated(n, T=0, x=None) == B.MOE_OK
    assert _gated(None) == B.MOE_EINVAL
    for bad in (dict(T=-1), dict(x=None), dict(h=None), dict(ldx=63), dict(ldh=(1 << 20) + 1), dict(x=FAKE + 1), dict(w=FAKE + 1),
                dict(gate=FAKE, ldg=64), dict(nw=FAKE), dict(y=FAKE * 2, ldy=64), dict(q=FAKE, ldq=64, s=FAKE), dict(c=FAKE + 1),
                dict(r=FAKE, ldr=63), dict(ldx=72, ldh=64), dict(r=FAKE * 2, ldr=72, h=FAKE * 2)):
        assert _gated(n, **bad) == B.MOE_EINVAL, bad
    assert _gated(B.gated_norm(64, normalize=False), w=FAKE) == B.MOE_EINVAL
    g = B.gated_norm(64, gate=B.GATE_SILU)
    assert _gated(g) == B.MOE_EINVAL and _gated(g, gate=FAKE, ldg=63) == B.MOE_EINVAL and _gated(g, gate=FAKE + 1, ldg=64) == B.MOE_EINVAL
    assert _gated(g, gate=FAKE, ldg=72, x=FAKE * 2) == B.MOE_EINVAL     # h over the gate, another stride
    row = B.gated_norm(64, gate=B.GATE_SILU, gate_per_row=True)
    assert _gated(row, gate=FAKE, ldg=0) == B.MOE_EINVAL
    nx = B.gated_norm(64, next_norm=True)
    assert _gated(nx) == B.MOE_EINVAL and _gated(nx, nw=FAKE + 1) == B.MOE_EINVAL
    assert _gated(nx, nw=FAKE, x=FAKE * 2, y=FAKE, ldy=72) == B.MOE_EINVAL    # y over h, another stride
    n8 = B.gated_norm(64, out8=B.OUT8_INT8, out8_group=32)
    assert _gated(n8) == B.MOE_EINVAL and _gated(n8, q=FAKE, ldq=64) == B.MOE_EINVAL
    assert _gated(n8, q=FAKE, ldq=63, s=FAKE) == B.MOE_EINVAL and _gated(n8, q=FAKE, ldq=64, s=FAKE + 2) == B.MOE_EINVAL
    for bad in (dict(eps=0.0), dict(eps=1e-39), dict(next_eps=-1.0), dict(eps=math.nan), dict(weight_offset=math.inf), dict(scale=math.nan),
                dict(next_offset=math.inf), dict(gate=3), dict(gate=-1), dict(out8=3)):
        assert _gated(B.gated_norm(64, **bad)) == B.MOE_EINVAL, bad
    for bad in (dict(H=0), dict(H=16385), dict(H=96, group=64), dict(H=96, group=48), dict(H=96, out8_group=64), dict(H=64, group=-32)):
        assert _gated(B.gated_norm(**bad)) == B.MOE_EUNSUPPORTED, bad
    for i, v in ((1, 3), (2, B.F16), (3, 2), (6, 2), (7, -1)):
        a = [getattr(n, f) for f, _ in B.MoeBlockNorm._fields_]
        a[i] = v
        assert _gated(B.MoeBlockNorm(*a)) == B.MOE_EINVAL, i


def test_gated_binding_checks_tensors():
    n = B.gated_norm(64, group=32, gate=B.GATE_SILU)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for kw in (dict(x=x.float()), dict(gate=x[:, :32]), dict(gate=x[:3]), dict(weight=torch.ones(31, dtype=torch.bfloat16)),
               dict(weight=torch.ones(32)), dict(h_out=x.half()), dict(channel_scale=x[0, :63]), dict(residual=x[:2]),
               dict(next_weight=x[0, :9]), dict(q=x, scales=torch.zeros(4)), dict()):
        a = dict(x=x, gate=x, h_out=torch.empty_like(x))
        a.update(kw)
        with pytest.raises(ValueError):  # (the last: every check passes; there is no CPU path)
            B.moe_gated_norm(n, a.pop("x"), 4, **a)
