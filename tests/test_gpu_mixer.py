"""GPU parity of the operators of a block's mixer half: the int8 projection, rotary positions, linear
attention with a decay for each head, the norm after a block, and a run of them together.

Every result is compared with a plain implementation in 64 bits (mixer_ref.py); the tolerances there are
bounds derived from the number formats."""
import math

import numpy as np
import pytest
import torch

from int4_grouped_gemm_router_amd import binding as B

from mixer_ref import gated_ref, int8_ref, linear_bound, linear_ref, rope_ref
from ops_ref import U32, half_step

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


def _close(got, want, err, dt, what):
    """got (of type dt) within the rounding of a value that is within err of want."""
    tol = half_step(dt, want.abs() + err) + err
    off = (got.cpu().double() - want).abs()
    assert (off <= tol).all(), f"{what}: {(off / tol).max():.3f} of its bound"


# ------------------------------------------------------------------ int8 projection

def _int8_case(T, N, K, dtype="bf16", bias=False, pad=0, ypad=0, extreme=False, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + N + K)
    x = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    if extreme:
        x.fill_(-128)
        w.fill_(-128)
        w[1::2] = 127
    xs, ws = torch.rand(T, generator=g) * 0.02 + 0.001, torch.rand(N, generator=g) * 0.002 + 0.0001
    b = torch.randn(N, generator=g) if bias else None
    dt = DT[dtype]
    xv = _wide(x, pad, 1, 3)[0]
    yv, yf = _wide(torch.zeros((T, N), dtype=dt), ypad, 2)
    work = B.project_int8_workspace(N, K, T)
    if work is not None:
        work.fill_(GUARD)
    B.moe_project_int8(w.cuda(), ws.cuda(), xv, xs.cuda(), yv, T, bias=None if b is None else b.cuda(), ws=work)
    torch.cuda.synchronize()
    y, err = int8_ref(w, ws, x, xs, b)
    _close(yv, y, err, dt, "y")
    assert _behind(yf, T, N)


INT8_CASES = [
    dict(T=1, N=1, K=64), dict(T=1, N=64, K=64), dict(T=1, N=2048, K=2048), dict(T=1, N=12288, K=2048, bias=True),
    dict(T=1, N=1000, K=8192), dict(T=2, N=65, K=128), dict(T=3, N=100, K=192, pad=16), dict(T=4, N=4096, K=4096),
    dict(T=15, N=513, K=320), dict(T=16, N=512, K=512), dict(T=17, N=512, K=2048, dtype="f16"), dict(T=31, N=257, K=64),
    dict(T=33, N=640, K=1088, dtype="f32", bias=True), dict(T=48, N=2000, K=2048, ypad=3), dict(T=64, N=64, K=4096),
    dict(T=65, N=300, K=448, ypad=8), dict(T=100, N=1023, K=960, dtype="f16", ypad=1), dict(T=127, N=129, K=576),
    dict(T=128, N=128, K=128), dict(T=200, N=2048, K=256), dict(T=255, N=255, K=64), dict(T=256, N=256, K=4160),
    dict(T=257, N=4097, K=192, dtype="f32"), dict(T=500, N=2000, K=4096, dtype="f16", bias=True, pad=64),
    dict(T=600, N=1536, K=2048, pad=32), dict(T=1000, N=2048, K=1024), dict(T=1025, N=6000, K=704, ypad=2),
    dict(T=2049, N=2304, K=512), dict(T=4096, N=4096, K=128), dict(T=5, N=300, K=65536), dict(T=300, N=320, K=16384),
    dict(T=3, N=1 << 18, K=64), dict(T=40000, N=48, K=64), dict(T=(1 << 18) + 37, N=16, K=64, ypad=2), dict(T=1, N=40, K=65536, extreme=True, dtype="f32"),
    dict(T=300, N=300, K=65536, extreme=True, dtype="f32"), dict(T=20, N=80, K=65536, extreme=True),
]


@pytest.mark.parametrize("c", INT8_CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_int8_matches_64_bits(c):
    _int8_case(**c)


def test_int8_reads_the_norms_rows():
    """moe_add_rmsnorm's 8-bit rows as they are: the product is that of the rows it was given, up to their rounding."""
    T, H, N = 70, 512, 300
    g = torch.Generator().manual_seed(4)
    x = torch.randn((T, H), generator=g).bfloat16()
    nw, w = (torch.rand(H, generator=g) + 0.5).bfloat16(), torch.randint(-127, 128, (N, H), generator=g, dtype=torch.int8)
    ws = torch.rand(N, generator=g) * 0.01
    n = B.norm(H, out8=B.OUT8_INT8)
    q, s = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty((T, 1), device="cuda")
    y = torch.empty((T, N), dtype=torch.float32, device="cuda")
    B.moe_add_rmsnorm(n, x.cuda(), nw.cuda(), T, q=q, scales=s)
    B.moe_project_int8(w.cuda(), ws.cuda(), q, s, y, T)
    want, err = int8_ref(w, ws, q.cpu(), s.cpu()[:, 0], None)
    _close(y, want, err, torch.float32, "y")


# ------------------------------------------------------------------ rotary positions

def _rope_case(T, q_heads, k_heads, D, rot, dtype="bf16", interleaved=False, inverse=False, inplace=False, pad=0, far=False,
               magnitude=1.0, positions=None, seed=0):
    g = torch.Generator().manual_seed(seed + T + 13 * D + rot)
    dt = DT[dtype]
    qkv = torch.randn((T, (q_heads + k_heads) * D), generator=g).to(dt)
    if positions is None:
        span = (1 << 31) - 1 if far else 5000
        positions = torch.randint(-span if far else 0, span, (T,), generator=g).to(torch.int32)
    rad, _ = B.rope_radians(rot, base=1e6)
    plan = B.rope(D, rot, dtype=dt, interleaved=interleaved, inverse=inverse, radians=rad, magnitude=magnitude)
    full_v, full = _wide(qkv, pad, 1)
    q, k = full_v[:, :q_heads * D], full_v[:, q_heads * D:] if k_heads else None
    want, err = rope_ref(qkv.view(T, -1, D), positions, torch.from_numpy(rad), rot, interleaved, magnitude, inverse)
    shape = lambda t, h: t.unflatten(1, (h, D))  # noqa: E731
    if inplace:
        B.moe_rope(plan, positions.cuda(), T, shape(q, q_heads), k=None if k is None else shape(k, k_heads))
        torch.cuda.synchronize()
        got = full_v
        assert _behind(full, T, qkv.shape[1])
    else:
        qo, qf = _wide(torch.zeros((T, q_heads * D), dtype=dt), pad, 2)
        ko, kf = _wide(torch.zeros((T, k_heads * D), dtype=dt), pad + 1, 2) if k_heads else (None, None)
        B.moe_rope(plan, positions.cuda(), T, shape(q, q_heads), k=None if k is None else shape(k, k_heads),
                   q_out=shape(qo, q_heads), k_out=None if ko is None else shape(ko, k_heads))
        torch.cuda.synchronize()
        assert _behind(qf, T, q_heads * D)
        assert torch.equal(full_v.cpu(), qkv)
        got = qo if ko is None else torch.cat([qo, ko], 1)
        assert ko is None or _behind(kf, T, k_heads * D)
    got = got.reshape(T, -1, D)
    _close(got, want, err, dt, "turned")
    assert torch.equal(got[..., rot:].cpu(), qkv.view(T, -1, D)[..., rot:])


ROPE_CASES = [
    dict(T=1, q_heads=1, k_heads=1, D=2, rot=2), dict(T=1, q_heads=16, k_heads=2, D=256, rot=64),
    dict(T=1, q_heads=8, k_heads=0, D=128, rot=128, interleaved=True), dict(T=5, q_heads=3, k_heads=2, D=10, rot=6),
    dict(T=5, q_heads=3, k_heads=1, D=10, rot=10, interleaved=True), dict(T=7, q_heads=5, k_heads=1, D=64, rot=30, pad=3),
    dict(T=7, q_heads=5, k_heads=3, D=65, rot=50, interleaved=True, pad=1), dict(T=33, q_heads=4, k_heads=4, D=80, rot=80),
    dict(T=33, q_heads=6, k_heads=2, D=96, rot=34, interleaved=True, dtype="f16"),
    dict(T=33, q_heads=6, k_heads=2, D=128, rot=128, dtype="f32"),
    dict(T=33, q_heads=6, k_heads=2, D=128, rot=126, dtype="f32", interleaved=True, pad=1),
    dict(T=50, q_heads=7, k_heads=1, D=128, rot=64, inplace=True), dict(T=50, q_heads=2, k_heads=1, D=33, rot=18, inplace=True),
    dict(T=50, q_heads=2, k_heads=1, D=33, rot=22, inplace=True, interleaved=True, pad=2, dtype="f32"),
    dict(T=40, q_heads=4, k_heads=2, D=64, rot=64, far=True, dtype="f32"),
    dict(T=40, q_heads=4, k_heads=2, D=64, rot=64, far=True, interleaved=True, dtype="f32"),
    dict(T=40, q_heads=4, k_heads=2, D=64, rot=32, inverse=True, magnitude=1.3),
    dict(T=9, q_heads=2, k_heads=1, D=1024, rot=1024), dict(T=9, q_heads=2, k_heads=1, D=1024, rot=2),
    # long calls: four heads a thread, head counts that four does not divide
    dict(T=2000, q_heads=32, k_heads=8, D=128, rot=128), dict(T=3000, q_heads=9, k_heads=2, D=128, rot=96, interleaved=True),
    dict(T=6001, q_heads=5, k_heads=0, D=72, rot=50), dict(T=6001, q_heads=3, k_heads=3, D=136, rot=100, inplace=True),
    dict(T=3000, q_heads=9, k_heads=2, D=128, rot=64, pad=1, dtype="f16"),
    dict(T=3001, q_heads=6, k_heads=1, D=128, rot=128, dtype="f32", interleaved=True),
]


@pytest.mark.parametrize("c", ROPE_CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_rope_matches_64_bits(c):
    _rope_case(**c)


def test_rope_every_quarter():
    """Angles around each eighth of a turn, both sides, to the last steps of the fixed point."""
    turn = 2 * math.pi
    rad = np.array([turn / 8, turn / 4, turn * (1 / 8 - 2.0 ** -33), turn * (1 / 2 - 2.0 ** -31), turn * 3 / 8 + 1e-9, 0.0,
                    -turn / 16, 5 * turn + 0.3])
    plan = B.rope(16, dtype=torch.float32, radians=rad)
    positions = torch.arange(-20, 21, dtype=torch.int32)
    x = torch.zeros((41, 1, 16))
    x[..., :8] = 1
    y = torch.empty((41, 1, 16), device="cuda")
    B.moe_rope(plan, positions.cuda(), 41, x.cuda(), q_out=y)
    angle = positions.double()[:, None] * torch.from_numpy(rad)
    for got, f in ((y[:, 0, :8], torch.cos), (y[:, 0, 8:], torch.sin)):
        assert ((got.cpu().double() - f(angle)).abs() <= 7.5 * U32 + angle.abs() * 2.0 ** -52).all()


def test_rope_inverse_undoes():
    T, H, D = 300, 4, 64
    x = torch.randn((T, H, D), device="cuda")
    p = torch.arange(T, dtype=torch.int32, device="cuda") * 977
    y, z = torch.empty_like(x), torch.empty_like(x)
    B.moe_rope(B.rope(D, dtype=torch.float32), p, T, x, q_out=y)
    B.moe_rope(B.rope(D, dtype=torch.float32, inverse=True), p, T, y, q_out=z)
    pair = (x[..., :32].abs() + x[..., 32:].abs()).double().repeat(1, 1, 2)
    assert ((z.double() - x.double()).abs() <= 2 * 9.5 * U32 * 2 * pair).all()  # twice the bound of one, whose pairs grow by sqrt 2 at most


# ------------------------------------------------------------------ linear attention

def _linear_inputs(T, Hk, Hv, dk, dv, per_token, seed, strong=0.0):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn((T, Hk, dk), generator=g) / math.sqrt(dk) for _ in range(2))
    v = torch.randn((T, Hv, dv), generator=g)
    decay = -torch.exp(torch.randn(Hv, generator=g) * 2 - 3)
    if per_token:
        decay = decay * torch.exp(torch.randn((T, Hv), generator=g))
        decay = torch.where(torch.rand((T, Hv), generator=g) < strong, decay * 300, decay)
    return q.bfloat16(), k.bfloat16(), v.bfloat16(), decay


def _view(t, pad):
    """[T, heads, dim] on the GPU in rows of heads * dim + pad."""
    T, H, D = t.shape
    return _wide(t.reshape(T, H * D), pad)[0].unflatten(1, (H, D))


def _linear_case(lengths, Hk=2, Hv=4, dk=64, dv=64, per_token=True, pad=0, behind=0, slots=None, inplace=False, scale=None,
                 step=False, seed=0, strong=0.0, decay=None, keep=True, start=True):
    n, L = len(lengths), sum(lengths)
    T = L + behind
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    q, k, v, g = _linear_inputs(T, Hk, Hv, dk, dv, per_token, seed + 3 * T + dk, strong)
    if decay is not None:
        g = decay(g)
    pool = torch.randn((n + 2, Hv, dk, dv), generator=torch.Generator().manual_seed(seed + 5))
    slots = list(range(n)) if slots is None else slots
    plan = B.linear_attention(Hk, Hv, dk, dv, scale=scale)
    o, of = _wide(torch.zeros((T, Hv * dv), dtype=torch.bfloat16), pad, 1)
    o = o.unflatten(1, (Hv, dv))
    full = of.clone()
    sin = pool.cuda() if start else None
    sout = (sin if inplace else torch.full((n + 1, Hv, dk, dv), 9.0, device="cuda")) if keep else None
    st = torch.tensor(slots, dtype=torch.int32, device="cuda") if start else None
    kw = dict(state_in=sin, slots_in=st, state_out=sout, slots_out=st if inplace and keep else None)
    args = (plan, _view(q, pad), _view(k, pad), _view(v, pad), g.cuda() if g.dim() == 1 else _wide(g, pad)[0], o)
    if step:
        B.moe_linear_attention_step(*args, T, **kw)
    else:
        ws = B.linear_attention_workspace(plan, n, T)
        if ws is not None:
            ws.fill_(GUARD)
        B.moe_linear_attention(*args, torch.from_numpy(cu).cuda(), T, ws=ws, **kw)
    torch.cuda.synchronize()
    starts = torch.stack([pool[s] if start and 0 <= s < n + 2 else torch.zeros_like(pool[0]) for s in slots])
    gt = g if g.dim() == 2 else g.expand(T, Hv)
    sc = dk ** -0.5 if scale is None else float(np.float32(scale))
    want, weight, states, sums = linear_ref(q, k, v, gt, starts, cu, sc)
    ro, rs = linear_bound(dk, max(lengths), not step)
    _close(o[:L], want[:L], ro * weight[:L], torch.bfloat16, "o")
    # rows behind the last sequence and values behind a row
    assert torch.equal(of.cpu()[L:], full.cpu()[L:]) and torch.equal(of.cpu()[:, Hv * dv:], full.cpu()[:, Hv * dv:])
    if L * Hv * dv >= 20000 and not step:
        # three roundings to bf16 (o's and the two operands'), each of 2^-8 / sqrt(3) at most in the mean
        rel = (o[:L].cpu().double() - want[:L]).norm() / want[:L].norm()
        assert rel <= 2.0 ** -8, rel
    if keep:
        got = sout.cpu().double()
        for i, s in enumerate(slots):
            if inplace and not 0 <= s < n + 2:
                continue
            a, b = got[s if inplace else i], states[i]
            assert ((a - b).abs() <= rs * sums[i] + U32 * b.abs() + 1e-37).all(), (i, ((a - b).abs() / (sums[i] + 1e-30)).max())
        if inplace:
            for s in set(range(n + 2)) - set(slots):
                assert torch.equal(sout[s].cpu(), pool[s])
        else:
            assert (sout[n] == 9.0).all()


LINEAR_CASES = [
    dict(lengths=[1]), dict(lengths=[2]), dict(lengths=[63]), dict(lengths=[64]), dict(lengths=[65]), dict(lengths=[200]),
    dict(lengths=[0]), dict(lengths=[0, 0, 5, 0]), dict(lengths=[0], behind=3), dict(lengths=[70], behind=70),
    dict(lengths=[1, 0, 63, 130, 0, 64, 3, 0], behind=9, pad=8), dict(lengths=[5] * 40), dict(lengths=[1] * 70),
    dict(lengths=[300], Hk=1, Hv=1, dk=8, dv=8), dict(lengths=[100, 30], Hk=1, Hv=3, dk=16, dv=24),
    dict(lengths=[90, 129], Hk=2, Hv=2, dk=96, dv=80, pad=16), dict(lengths=[190], Hk=2, Hv=4, dk=128, dv=128),
    dict(lengths=[190, 11], Hk=1, Hv=2, dk=256, dv=256), dict(lengths=[130], Hk=1, Hv=2, dk=200, dv=40),
    dict(lengths=[130], Hk=1, Hv=1, dk=40, dv=248), dict(lengths=[77], Hk=4, Hv=4, dk=32, dv=128),
    dict(lengths=[150, 60], per_token=False, Hk=3, Hv=3), dict(lengths=[1500], Hk=1, Hv=2, dk=64, dv=64),
    dict(lengths=[700, 1, 900, 64], Hk=1, Hv=2, dk=128, dv=64), dict(lengths=[513, 1023], Hk=1, Hv=1, dk=64, dv=128),
    # states: unknown slots, one state read by several, in place, none at all
    dict(lengths=[70, 3, 0, 65], slots=[-1, 2, 99, 2]), dict(lengths=[70, 3, 0, 65], slots=[5, 1, 0, 2], inplace=True),
    dict(lengths=[700, 3, 400], slots=[1, -1, 3], inplace=True, Hv=2), dict(lengths=[100, 20], start=False),
    dict(lengths=[100, 20], keep=False), dict(lengths=[600, 20], start=False, keep=False),
    dict(lengths=[128], scale=1.0, strong=0.1), dict(lengths=[400], scale=-0.5, strong=0.5), dict(lengths=[70], scale=0.0),
    # many sequences, short ones beside long ones, in place and not
    dict(lengths=[1] * 20 + [300] + [8, 9, 0, 7] + [2] * 9), dict(lengths=[5, 600, 0, 8, 0, 9, 1, 1, 64, 3], inplace=True, Hv=2),
    dict(lengths=[0] * 9), dict(lengths=[0] * 9, behind=2, inplace=True), dict(lengths=[3] * 12, slots=[-1, 13] + [4] * 10, behind=5),
    dict(lengths=[20] * 100, Hk=1, Hv=2, dk=32, dv=64), dict(lengths=[9] * 28, dk=32, dv=72, slots=[27] * 3 + [-1] * 25), dict(lengths=[0, 11, 0, 0, 9, 200, 8], Hk=1, Hv=2, inplace=True), dict(lengths=[0, 33, 8, 15, 1, 40] * 30, Hk=1, Hv=2, dk=64, dv=32, inplace=True),
    # 128 columns of a state a block, one window and several
    dict(lengths=[1, 150, 39], Hk=390, Hv=780, dk=16, dv=72), dict(lengths=[1000, 0, 700, 621], Hk=16, Hv=64, dk=16, dv=80, slots=[3, 1, 0, 5], inplace=True),
    dict(lengths=[30, 1300, 991], Hk=32, Hv=64, dk=72, dv=72), dict(lengths=[1900, 700], Hk=60, Hv=60, dk=24, dv=136, per_token=False, behind=3),
    dict(lengths=[8] * 70 + [400], Hk=1, Hv=1, dk=32, dv=32), dict(lengths=[1] * 130, Hk=1, Hv=2, dk=40, dv=72, per_token=False),
]


@pytest.mark.parametrize("c", LINEAR_CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_linear_matches_64_bits(c):
    _linear_case(**c)


@pytest.mark.parametrize("n,more", [(1, {}), (3, dict(pad=8)), (9, dict(Hk=1, Hv=3, dk=40, dv=24)), (33, dict(dk=128, dv=128)),
                                    (5, dict(Hk=1, Hv=2, dk=256, dv=256)), (4, dict(Hk=1, Hv=1, dk=8, dv=8)),
                                    (6, dict(per_token=False)), (6, dict(slots=[4, -1, 4, 99, 0, 1])),
                                    (6, dict(slots=[7, 1, 0, 5, 3, 2], inplace=True)), (3, dict(start=False)),
                                    (3, dict(keep=False)), (3, dict(start=False, keep=False)), (300, dict(Hk=1, Hv=1, dk=64, dv=32))])
def test_linear_step_matches_64_bits(n, more):
    _linear_case([1] * n, step=True, **more)


def test_linear_forgets_at_minus_infinity():
    """A decay of -inf drops everything before its token and nothing after it; very strong ones lose no precision of
    what follows."""
    def cut(value):
        def f(g):
            g = g.clone()
            g[37], g[64], g[100, 1], g[101, 1] = value, value, value, value
            return g
        return f
    for value in (-math.inf, -1e30, -500.0, -90.0):
        _linear_case([30, 120, 40], decay=cut(value))
    _linear_case([1] * 40, step=True, decay=lambda g: torch.full_like(g, -math.inf))


def test_linear_growth():
    """Positive log decays are allowed as long as the results stay in range."""
    _linear_case([100], decay=lambda g: g.abs() * 0.3)


def test_linear_nan_stays_in_its_head_and_sequence():
    T, H, D = 150, 2, 64
    q, k, v, g = _linear_inputs(T, H, H, D, D, True, 3)
    clean = [t.cuda() for t in (q, k, v)]
    plan, cu = B.linear_attention(H, H, D, D), torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda")
    ws = B.linear_attention_workspace(plan, 2, T)

    def run(q, k, v, g):
        o, S = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((2, H, D, D), device="cuda")
        B.moe_linear_attention(plan, q, k, v, g, o, cu, T, state_out=S, ws=ws)
        return o.cpu(), S.cpu()
    o0, S0 = run(*clean, g.cuda())
    bad = g.clone()
    bad[40, 0] = math.nan
    o1, S1 = run(*clean, bad.cuda())
    assert torch.equal(o1[:, 1], o0[:, 1]) and torch.equal(o1[70:], o0[70:]) and torch.equal(o1[:40, 0], o0[:40, 0])
    assert o1[40:70, 0].isnan().all() and S1[0, 0].isnan().all()
    assert torch.equal(S1[1], S0[1]) and torch.equal(S1[0, 1], S0[0, 1])


@pytest.mark.parametrize("D,Hv,value", [(64, 2, math.nan), (64, 2, math.inf), (128, 2, -math.inf), (40, 1, math.nan), (256, 1, math.inf), (72, 740, math.nan)])
def test_linear_not_finite_values_reach_no_earlier_token(D, Hv, value):
    """A NaN or infinity of one token's value, key or query reaches that token and, but for the query, its later ones,
    never an earlier token, another sequence or (a value) another column."""
    T, at = 200, 75
    q, k, v, g = _linear_inputs(T, Hv, Hv, D, D, True, 17)
    plan, cu = B.linear_attention(Hv, Hv, D, D), torch.tensor([0, 50, 150, 200], dtype=torch.int32, device="cuda")
    ws = B.linear_attention_workspace(plan, 3, T)

    def run(q, k, v):
        o, S = torch.empty((T, Hv, D), dtype=torch.bfloat16, device="cuda"), torch.empty((3, Hv, D, D), device="cuda")
        B.moe_linear_attention(plan, q.cuda(), k.cuda(), v.cuda(), g.cuda(), o, cu, T, state_out=S, ws=ws)
        return o.cpu(), S.cpu()
    o0, S0 = run(q, k, v)
    for which in range(3):
        bad = [t.clone() for t in (q, k, v)]
        bad[which][at, 0, 5] = value
        o, S = run(*bad)
        same = torch.ones((T, Hv, D), dtype=torch.bool)
        if which == 0:
            same[at, 0] = False
        elif which == 1:
            same[at:150, 0] = False
        else:
            same[at:150, 0, 5] = False
        assert torch.equal(o[same], o0[same]), which
        assert not o[~same].isfinite().any(), which
        assert torch.equal(S[[0, 2]], S0[[0, 2]])
        if which == 0:
            assert torch.equal(S, S0)
        elif which == 2:
            assert not S[1, 0, :, 5].isfinite().any() and torch.equal(S[1, 0, :, :5], S0[1, 0, :, :5])


def test_linear_offsets_out_of_order_stay_in_range():
    """What cu_seqlens holds is limited to 0..T and to ends that are not before their beginnings: rows of no sequence
    are left alone, and nothing outside the buffers is touched."""
    T, H, D = 90, 1, 32
    q, k, v, g = (t.cuda() for t in _linear_inputs(T, H, H, D, D, True, 8))
    plan = B.linear_attention(H, H, D, D)
    for cu in ([0, 40, 500], [-7, 30, 1 << 30], [0, 60, 20, 2000000000], [80, 10, -5]):
        n = len(cu) - 1
        o = torch.full((T + 4, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
        S = torch.full((n + 1, H, D, D), 3.0, device="cuda")
        B.moe_linear_attention(plan, q, k, v, g, o, torch.tensor(cu, dtype=torch.int32, device="cuda"), T, state_out=S[:n],
                               ws=B.linear_attention_workspace(plan, n, T))
        torch.cuda.synchronize()
        assert (o[T:] == 3.0).all() and (S[n] == 3.0).all()


def test_linear_prompt_then_steps_is_one_prompt():
    """A prompt in two pieces and then single tokens, states kept in one pool, against the whole at once."""
    T, Hk, Hv, D = 140, 2, 4, 64
    q, k, v, g = _linear_inputs(T, Hk, Hv, D, D, True, 21)
    dev = [t.cuda() for t in (q, k, v, g)]
    plan = B.linear_attention(Hk, Hv, D, D)
    pool = torch.full((3, Hv, D, D), 5.0, device="cuda")
    o = torch.empty((T, Hv, D), dtype=torch.bfloat16, device="cuda")
    none, one = (torch.tensor([s], dtype=torch.int32, device="cuda") for s in (-1, 1))
    at = 0
    for m in (70, 50):
        part = [t[at:at + m] for t in dev]
        B.moe_linear_attention(plan, *part, o[at:at + m], torch.tensor([0, m], dtype=torch.int32, device="cuda"), m,
                               state_in=pool, slots_in=none if at == 0 else one, state_out=pool, slots_out=one,
                               ws=B.linear_attention_workspace(plan, 1, m))
        at += m
    for t in range(at, T):
        B.moe_linear_attention_step(plan, *[x[t:t + 1] for x in dev], o[t:t + 1], 1, state_in=pool, slots_in=one,
                                    state_out=pool, slots_out=one)
    torch.cuda.synchronize()
    want, weight, states, sums = linear_ref(q, k, v, g, torch.zeros((1, Hv, D, D)), [0, T], D ** -0.5)
    ro, rs = linear_bound(D, T, True)
    _close(o, want, (ro + 100 * U32) * weight, torch.bfloat16, "o")
    assert ((pool[1].cpu().double() - states[0]).abs() <= (rs + 100 * U32) * sums[0]).all()
    assert (pool[0] == 5.0).all() and (pool[2] == 5.0).all()


# ------------------------------------------------------------------ the norm after a block

def _gated_case(T, H, group=0, dtype="bf16", weight=None, normalize=True, weighted=True, gate=0, row=False, residual=False,
                channel=False, scale=1.0, following=False, out8=B.OUT8_NONE, out8_group=0, offset=0.0, pad=0, h=True, y=True,
                inplace=None, seed=0, eps=1e-6, x=None):
    gen = torch.Generator().manual_seed(seed + 31 * T + H)
    dt, wt = DT[dtype], DT[weight or dtype]
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x = (rnd(T, H) * torch.exp(rnd(T, 1)) if x is None else x).to(dt)
    w = (torch.rand(group or H, generator=gen) + 0.5 - offset).to(wt) if normalize and weighted else None
    z = (rnd(T, 1 if row else H) * 3).to(dt) if gate else None
    c = (torch.rand(H, generator=gen) + 0.5).to(wt) if channel else None
    r = (rnd(T, H) * 2).to(dt) if residual else None
    nw = (torch.rand(H, generator=gen) + 0.5 - offset).to(wt) if following else None
    n = B.gated_norm(H, dtype=dt, weight_dtype=wt, normalize=normalize, group=group, eps=eps, weight_offset=offset, gate=gate,
                     gate_per_row=row, scale=scale, next_norm=following, next_eps=eps, next_offset=offset, out8=out8,
                     out8_group=out8_group)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    xv, xf = _wide(x, pad, 1)
    rv = _wide(r, pad, 1)[0] if residual else None
    zv = None if z is None else _wide(z, pad, 1)[0]
    hv, hf = _wide(torch.zeros_like(x), pad, 2)
    yv, yf = _wide(torch.zeros_like(x), pad, 2)
    if inplace:
        hv = {"x": xv, "residual": rv, "gate": zv}[inplace]
    q = s = qf = None
    G = H // out8_group if out8_group else 1
    if out8:
        q, qf = _wide(torch.zeros((T, H), dtype=torch.uint8), pad, 2, GUARD)
        s = torch.full((T + 1, G), -1.0, device="cuda")
    B.moe_gated_norm(n, xv, T, weight=dev(w), gate=zv, channel_scale=dev(c), residual=rv, next_weight=dev(nw),
                     h_out=hv if h else None, y=yv if following and y else None, q=q, scales=s)
    torch.cuda.synchronize()
    cc = dict(normalize=normalize, group=group, offset=offset, eps=float(np.float32(eps)), gate=gate,
              scale=float(np.float32(scale)))
    v, verr, yw, yerr = gated_ref(x, cc, w, z, c, r, nw)
    if h:
        _close(hv, v, verr, dt, "h")
        assert inplace or _behind(hf, T, H)
    if following and y:
        _close(yv, yw, yerr, dt, "y")
        assert _behind(yf, T, H)
    if out8:
        if following:
            v, verr = yw, yerr
        Q = 127.0 if out8 == B.OUT8_INT8 else 448.0
        vg, eg = v.reshape(T, G, -1), verr.reshape(T, G, -1)
        sref, serr = vg.abs().amax(2) / Q, eg.amax(2) / Q
        sc = s.cpu().double()
        assert ((sc[:T] - sref).abs() <= serr + 2 * U32 * sref + 2.0 ** -149).all()
        assert (sc[T:] == -1).all()
        assert _behind(qf, T, H, GUARD)
        live = sref > 1e-30
        d = torch.where(live, sref, torch.ones_like(sref))[:, :, None]
        want = torch.where(live[:, :, None], vg / d, torch.zeros_like(vg))
        off = torch.where(live[:, :, None], (eg + want.abs() * serr[:, :, None]) / d, torch.zeros_like(vg)) + 4 * U32 * want.abs()
        if out8 == B.OUT8_INT8:
            got = q.cpu().view(torch.int8).double().reshape(vg.shape)
            assert (got.abs() <= 127).all()
            step = 0.5
        else:
            got = q.cpu().contiguous().view(torch.float8_e4m3fn).double().reshape(vg.shape)
            step = (want.abs() * 2.0 ** -4).clamp(min=2.0 ** -10)  # half a step: 2^-4 relative, 2^-10 below 2^-6
        assert (((got - want).abs() <= step + off) | ~live[:, :, None]).all()


GATED_CASES = [
    dict(T=1, H=4096, group=128, gate=1, out8=B.OUT8_INT8), dict(T=300, H=2048, group=128, gate=2), dict(T=1, H=1), dict(T=5, H=7),
    dict(T=9, H=63, residual=True, following=True), dict(T=3, H=1537, gate=1, residual=True, following=True, pad=3),
    dict(T=3, H=128, group=32, gate=1), dict(T=3, H=128, group=128), dict(T=3, H=64, group=64, gate=2), dict(T=2, H=256, group=256),
    dict(T=33, H=512, group=64, gate=1, dtype="f16", weight="f32"), dict(T=33, H=1024, group=256, gate=1, dtype="f32"),
    dict(T=33, H=768, group=256, residual=True, channel=True, scale=0.3, following=True, out8=B.OUT8_E4M3, out8_group=128),
    dict(T=700, H=2048, residual=True, following=True, out8=B.OUT8_INT8, channel=True, scale=0.5, offset=1.0),
    dict(T=40, H=1024, normalize=False, gate=2, row=True, residual=True, following=True),
    dict(T=40, H=1000, normalize=False, gate=1, row=True, residual=True, pad=1), dict(T=40, H=1000, normalize=False, scale=2.0),
    dict(T=40, H=1024, weighted=False, group=128, scale=128 ** -0.5), dict(T=40, H=333, weighted=False, out8=B.OUT8_E4M3),
    dict(T=20, H=2048, gate=1, residual=True, inplace="x"), dict(T=20, H=2048, gate=1, residual=True, following=True, inplace="residual"),
    dict(T=20, H=1111, gate=2, residual=True, following=True, inplace="gate", pad=2),
    dict(T=20, H=512, residual=True, following=True, h=False), dict(T=20, H=512, out8=B.OUT8_INT8, h=False),
    dict(T=20, H=512, residual=True, following=True, y=False, out8=B.OUT8_INT8, out8_group=32),
    dict(T=3, H=4096, gate=1, residual=True, following=True, channel=True), dict(T=3, H=8192, gate=1, residual=True, following=True),
    dict(T=3, H=8200, gate=1, residual=True, following=True, channel=True, pad=5), dict(T=5, H=16384, group=256, gate=1, residual=True, following=True, out8=B.OUT8_INT8),
    dict(T=3, H=16383, residual=True, following=True, out8=B.OUT8_E4M3), dict(T=3, H=16384, dtype="f32", gate=2, residual=True, following=True, channel=True),
    dict(T=3, H=5000, dtype="f32", weight="f32", gate=1, out8=B.OUT8_INT8), dict(T=3, H=5120, group=64, dtype="f16", gate=1, out8=B.OUT8_E4M3, out8_group=256),
    dict(T=5000, H=96, group=32, gate=1, residual=True, following=True), dict(T=3000, H=2048, group=128, gate=1, out8=B.OUT8_INT8, pad=8),
    dict(T=2500, H=4096, residual=True, following=True),
]


@pytest.mark.parametrize("c", GATED_CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_gated_norm_matches_64_bits(c):
    _gated_case(**c)


def test_gated_norm_zero_rows_and_far_gates():
    """Rows of zeros give zeros and scales of 0; gates far on both sides saturate."""
    H = 256
    x = torch.randn((6, H))
    x[2] = 0
    _gated_case(6, H, x=x, group=64, out8=B.OUT8_INT8)
    n = B.gated_norm(H, dtype=torch.float32, normalize=False, gate=B.GATE_SILU, out8=B.OUT8_INT8)
    z = torch.tensor([-1e30, -200.0, -100.0, -80.0, 80.0, 200.0, 1e30, 0.0]).repeat(H // 8)[None].cuda()
    h, q, s = torch.empty((1, H), device="cuda"), torch.empty((1, H), dtype=torch.int8, device="cuda"), torch.empty((1, 1), device="cuda")
    B.moe_gated_norm(n, torch.ones((1, H), device="cuda"), 1, gate=z, h_out=h, q=q, scales=s)
    zd = z.cpu().double()
    want = zd * torch.sigmoid(zd)
    assert ((h.cpu().double() - want).abs() <= 12 * U32 * want.abs() + 2.0 ** -126 * 200).all()
    m = B.gated_norm(H, normalize=False, out8=B.OUT8_INT8)
    q.fill_(9)
    B.moe_gated_norm(m, torch.zeros((1, H), dtype=torch.bfloat16, device="cuda"), 1, q=q, scales=s)
    assert (q == 0).all() and (s == 0).all()


def test_gated_norm_nan_and_infinity_stay_in_their_rows():
    H = 512
    x = torch.randn((8, H)).bfloat16()
    g = torch.randn((8, H)).bfloat16()
    n = B.gated_norm(H, group=128, gate=B.GATE_SIGMOID, out8=B.OUT8_INT8, out8_group=128)

    def run(x, g):
        h, q, s = torch.empty_like(x.cuda()), torch.empty((8, H), dtype=torch.int8, device="cuda"), torch.empty((8, 4), device="cuda")
        B.moe_gated_norm(n, x.cuda(), 8, gate=g.cuda(), h_out=h, q=q, scales=s)
        return h.cpu(), q.cpu(), s.cpu()
    a = run(x, g)
    x2, g2 = x.clone(), g.clone()
    x2[3, 130] = math.nan
    x2[4, 5] = math.inf
    g2[6, 300] = math.nan
    b = run(x2, g2)
    for i in (0, 1, 2, 5, 7):
        assert all(torch.equal(p[i], q[i]) for p, q in zip(a, b))
    assert b[0][3, 128:256].isnan().all() and torch.equal(b[0][3, :128], a[0][3, :128]) and b[2][3, 1].isnan()
    assert b[0][4, 5].isnan() and (b[0][4, 6:128] == 0).all()
    assert b[0][6, 300].isnan() and (b[1][6, 256:384] == 0).all()


# ------------------------------------------------------------------ together

class _Mixer:
    """The mixer half of a block, as a program holds it: norm to int8, one projection into queries, keys, values, gates
    and decays, rotary positions, linear attention, the heads' norm with its gate to int8, the output projection, and the
    residual add with the next norm."""

    def __init__(self, T, seqs, H=512, Hk=2, Hv=4, D=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.H, self.Hk, self.Hv, self.D, self.n = T, H, Hk, Hv, D, len(seqs)
        self.widths = [Hk * D, Hk * D, Hv * D, Hv * D]
        N = sum(self.widths)
        q8 = lambda n, k: torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int8)  # noqa: E731
        self.w_in, self.w_out = q8(N, H), q8(H, Hv * D)
        self.s_in, self.s_out = torch.rand(N, generator=g) * 2e-4, torch.rand(H, generator=g) * 2e-4
        self.norm_w, self.next_w = ((torch.rand(H, generator=g) + 0.5).bfloat16() for _ in range(2))
        self.head_w = (torch.rand(D, generator=g) + 0.5).bfloat16()
        self.x, self.res = (torch.randn((T, H), generator=g).bfloat16() for _ in range(2))
        self.decay = -torch.rand((T, Hv), generator=g) * 0.2
        self.positions = torch.cat([torch.arange(L) for L in seqs]).to(torch.int32)
        self.cu = torch.tensor([0, *np.cumsum(seqs)], dtype=torch.int32)
        self.plans = (B.norm(H, out8=B.OUT8_INT8), B.rope(D, D // 2), B.linear_attention(Hk, Hv, D, D),
                      B.gated_norm(Hv * D, group=D, gate=B.GATE_SILU, out8=B.OUT8_INT8),
                      B.gated_norm(H, normalize=False, scale=0.5, next_norm=True))

    def to_gpu(self):
        names = ("w_in", "w_out", "s_in", "s_out", "norm_w", "next_w", "head_w", "x", "res", "decay", "positions", "cu")
        self.d = {n: getattr(self, n).cuda() for n in names}
        T, H, W = self.T, self.H, self.Hv * self.D
        new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.b = dict(q8=new(T, H, dtype=torch.int8), s8=new(T, 1, dtype=torch.float32), h=new(T, H), qkvg=new(T, sum(self.widths)),
                      o=new(T, W), o8=new(T, W, dtype=torch.int8), os=new(T, 1, dtype=torch.float32), z=new(T, H), h2=new(T, H),
                      y=new(T, H), S=new(self.n, self.Hv, self.D, self.D, dtype=torch.float32))
        self.ws = (B.project_int8_workspace(sum(self.widths), H, T), B.linear_attention_workspace(self.plans[2], self.n, T),
                   B.project_int8_workspace(H, W, T))
        return self

    def run(self):
        d, b, T, D = self.d, self.b, self.T, self.D
        norm, rope, lin, heads, block = self.plans
        B.moe_add_rmsnorm(norm, d["x"], d["norm_w"], T, residual=d["res"], h_out=b["h"], q=b["q8"], scales=b["s8"])
        B.moe_project_int8(d["w_in"], d["s_in"], b["q8"], b["s8"], b["qkvg"], T, ws=self.ws[0])
        q, k, v, z = b["qkvg"].split(self.widths, 1)
        q, k, v = q.unflatten(1, (self.Hk, D)), k.unflatten(1, (self.Hk, D)), v.unflatten(1, (self.Hv, D))
        B.moe_rope(rope, d["positions"], T, q, k=k)
        B.moe_linear_attention(lin, q, k, v, d["decay"], b["o"], d["cu"], T, state_out=b["S"], ws=self.ws[1])
        B.moe_gated_norm(heads, b["o"], T, weight=d["head_w"], gate=z, q=b["o8"], scales=b["os"])
        B.moe_project_int8(d["w_out"], d["s_out"], b["o8"], b["os"], b["z"], T, ws=self.ws[2])
        B.moe_gated_norm(block, b["z"], T, residual=b["h"], next_weight=d["next_w"], h_out=b["h2"], y=b["y"])

    def outputs(self):
        torch.cuda.synchronize()
        return {n: t.cpu().clone() for n, t in self.b.items()}

    def check(self, got):
        """Each step against 64 bits on what the step before it left."""
        T, D = self.T, self.D
        y, err = int8_ref(self.w_in, self.s_in, got["q8"], got["s8"][:, 0], None)
        q, k, v, z = got["qkvg"].split(self.widths, 1)
        yq, yk, yv, yz = y.split(self.widths, 1)
        eq, ek, ev, ez = err.split(self.widths, 1)
        _close(v, yv, ev, torch.bfloat16, "v")
        _close(z, yz, ez, torch.bfloat16, "gate")
        rad = torch.from_numpy(B.rope_radians(D // 2)[0])
        for t, w, e, h in ((q, yq, eq, self.Hk), (k, yk, ek, self.Hk)):
            # turned after one rounding to bf16: twice half a step of the pair
            turned, terr = rope_ref(w.reshape(T, h, D), self.positions, rad, D // 2, False)
            a = (half_step(torch.bfloat16, w) + e).reshape(T, h, D)
            half = D // 4
            pair = a[..., :half] + a[..., half:2 * half]
            a[..., :2 * half] = torch.cat([pair, pair], 2)
            _close(t.reshape(T, h, D), turned, terr + a, torch.bfloat16, "turned")
        start = torch.zeros((self.n, self.Hv, D, D))
        o, weight, S, sums = linear_ref(q.reshape(T, self.Hk, D), k.reshape(T, self.Hk, D), v.reshape(T, self.Hv, D), self.decay,
                                        start, self.cu.tolist(), D ** -0.5)
        ro, rs = linear_bound(D, T, True)
        _close(got["o"].reshape(T, self.Hv, D), o, ro * weight, torch.bfloat16, "o")
        assert ((got["S"].double() - S).abs() <= rs * sums + 1e-37).all()
        c = dict(normalize=True, group=D, offset=0.0, eps=float(np.float32(1e-6)), gate=1, scale=1.0)
        u, uerr, _, _ = gated_ref(got["o"], c, self.head_w, z)
        s = got["os"].double()
        assert ((got["o8"].double() * s - u).abs() <= s * (0.5 + 127 * 6 * U32) + uerr).all()
        y, err = int8_ref(self.w_out, self.s_out, got["o8"], got["os"][:, 0], None)
        _close(got["z"], y, err, torch.bfloat16, "z")
        c = dict(normalize=False, group=0, offset=0.0, eps=float(np.float32(1e-6)), gate=0, scale=0.5)
        h2, herr, y, yerr = gated_ref(got["z"], c, residual=got["h"], next_weight=self.next_w)
        _close(got["h2"], h2, herr, torch.bfloat16, "h2")
        _close(got["y"], y, yerr, torch.bfloat16, "y")


@pytest.mark.parametrize("seqs", [[1], [3, 1, 1], [40, 90], [300, 0, 25]], ids=str)
def test_mixer_together(seqs):
    m = _Mixer(sum(seqs), seqs).to_gpu()
    m.run()
    m.check(m.outputs())


def test_mixer_in_graphs_and_on_streams():
    """Captured graphs, eager work between their replays, another stream: the same bits as the eager run."""
    ms = [_Mixer(sum(s), s, seed=i).to_gpu() for i, s in enumerate(([200, 13], [7, 90]))]
    want = []
    for m in ms:
        m.run()
        want.append(m.outputs())
    # both graphs share one set of workspaces, as steps of one program that run one after the other do
    for i in range(3):
        a = ms[0].ws[i]
        if a is not None and ms[1].ws[i] is not None:
            big = max(a, ms[1].ws[i], key=lambda t: t.numel())
            for m in ms:
                m.ws = tuple(big if j == i else w for j, w in enumerate(m.ws))
    graphs = []
    for m in ms:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.run()
        graphs.append(g)
    for turn in range(4):
        for m, g, w in zip(ms, graphs, want):
            for n, t in m.b.items():
                t.fill_(3)
            if turn % 2:
                torch.cuda.synchronize()
            g.replay()
            got = m.outputs()
            assert all(torch.equal(got[n], w[n]) for n in w), turn
            (torch.ones(1000, device="cuda") * 2).sum().item()
    stream = torch.cuda.Stream()
    for n, t in ms[0].b.items():
        t.fill_(3)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ms[0].run()
    got = ms[0].outputs()
    assert all(torch.equal(got[n], want[0][n]) for n in want[0])


def test_rows_past_two_to_the_31st():
    """Rows a million elements apart, so that their offsets pass 32 bits: the same as rows side by side, bit for bit."""
    ld, T = 1 << 20, 2100
    g = torch.Generator().manual_seed(8)
    far = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")
    assert (T - 1) * ld > 1 << 31

    def spread(t, at):
        """t's rows in columns `at` on of `far`."""
        v = far[:, at:at + t.shape[1]]
        v.copy_(t)
        return v
    Hk, Hv, D = 1, 2, 64
    q, k, v, decay = (t.cuda() for t in _linear_inputs(T, Hk, Hv, D, D, True, 5))
    plan, cu = B.linear_attention(Hk, Hv, D, D), torch.tensor([0, 700, T], dtype=torch.int32, device="cuda")
    ws = B.linear_attention_workspace(plan, 2, T)
    o = torch.empty((T, Hv, D), dtype=torch.bfloat16, device="cuda")
    B.moe_linear_attention(plan, q, k, v, decay, o, cu, T, ws=ws)
    fo = far[:, 4096:4096 + Hv * D]
    B.moe_linear_attention(plan, spread(q.flatten(1), 0), spread(k.flatten(1), 1024), spread(v.flatten(1), 2048), decay, fo, cu, T,
                           ws=ws)
    assert torch.equal(fo, o.flatten(1))
    B.moe_linear_attention_step(plan, q, k, v, decay, o, T)
    B.moe_linear_attention_step(plan, far[:, :Hk * D], far[:, 1024:1024 + Hk * D], far[:, 2048:2048 + Hv * D], decay, fo, T)
    assert torch.equal(fo, o.flatten(1))

    rope, pos = B.rope(D), torch.arange(T, dtype=torch.int32, device="cuda")
    y = torch.empty_like(v)
    B.moe_rope(rope, pos, T, v, q_out=y)
    B.moe_rope(rope, pos, T, far[:, 2048:2048 + Hv * D])
    assert torch.equal(far[:, 2048:2048 + Hv * D], y.flatten(1))

    H = 128
    n = B.gated_norm(H, gate=B.GATE_SILU, next_norm=True)
    x, z, w = (torch.randn(s, generator=g).bfloat16().cuda() for s in ((T, H), (T, H), (H,)))
    h, y = torch.empty_like(x), torch.empty_like(x)
    B.moe_gated_norm(n, x, T, weight=w, gate=z, residual=x, next_weight=w, h_out=h, y=y)
    fh, fy = far[:, 8192:8192 + H], far[:, ld - H:]
    xf = spread(x, 3)
    B.moe_gated_norm(n, xf, T, weight=w, gate=spread(z, 5000), residual=xf, next_weight=w, h_out=fh, y=fy)
    assert torch.equal(fh, h) and torch.equal(fy, y)

    x8, w8 = (torch.randint(-128, 128, s, generator=g, dtype=torch.int8).cuda() for s in ((T, 256), (48, 256)))
    xs, wsc = torch.rand(T, generator=g).cuda(), torch.rand(48, generator=g).cuda()
    y = torch.empty((T, 48), dtype=torch.bfloat16, device="cuda")
    B.moe_project_int8(w8, wsc, x8, xs, y, T)
    far8 = torch.as_strided(far.view(torch.int8), (2 * T, 256), (ld, 1))  # (rows of a million bytes)
    far8[T:].copy_(x8)
    far8[:T].copy_(x8)
    y2 = torch.empty((2 * T, 48), dtype=torch.bfloat16, device="cuda")
    B.moe_project_int8(w8, wsc, far8, xs.repeat(2), y2, 2 * T)
    assert torch.equal(y2[:T], y) and torch.equal(y2[T:], y)
    fy = far[:, 1 << 19:(1 << 19) + 48]
    B.moe_project_int8(w8, wsc, x8, xs, fy, T)
    assert torch.equal(fy, y)


def test_linear_states_past_two_to_the_31st():
    """Slots at the end of a pool of more than 2^31 values: the same as in a small pool, bit for bit, in place."""
    Hk, Hv, D, n = 2, 16, 128, 8200
    assert n * Hv * D * D > 1 << 31
    pool = torch.empty((n, Hv, D, D), device="cuda")
    start = torch.randn((2, Hv, D, D), generator=torch.Generator().manual_seed(2)).cuda()
    plan = B.linear_attention(Hk, Hv, D, D)
    slots = torch.tensor([n - 1, n - 3], dtype=torch.int32, device="cuda")
    for T, cu in ((2, None), (50, [0, 20, 50]), (1400, [0, 1390, 1400])):
        q, k, v, g = (t.cuda() for t in _linear_inputs(T, Hk, Hv, D, D, True, T))
        small, o, o2 = start.clone(), torch.empty_like(v), torch.empty_like(v)
        pool[n - 1], pool[n - 3] = start[0], start[1]
        if cu is None:
            B.moe_linear_attention_step(plan, q, k, v, g, o, T, state_in=small, state_out=small)
            B.moe_linear_attention_step(plan, q, k, v, g, o2, T, state_in=pool, slots_in=slots, state_out=pool, slots_out=slots)
        else:
            cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
            ws = B.linear_attention_workspace(plan, 2, T)
            B.moe_linear_attention(plan, q, k, v, g, o, cu, T, state_in=small, state_out=small, ws=ws)
            B.moe_linear_attention(plan, q, k, v, g, o2, cu, T, state_in=pool, slots_in=slots, state_out=pool, slots_out=slots, ws=ws)
        assert torch.equal(o, o2) and torch.equal(pool[n - 1], small[0]) and torch.equal(pool[n - 3], small[1])
        assert not torch.equal(small, start)
