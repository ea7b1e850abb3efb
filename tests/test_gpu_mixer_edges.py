"""GPU tests of the operators of a block's mixer half where the other ones do not go: linear attention's edge values in
calls of several windows (states passed from one to the next), workspaces that captured graphs share, prompts followed by
single tokens out of one pool of states, and infinite gates.

Compared with the plain implementation in 64 bits (mixer_ref.py)."""
import math

import pytest
import torch

import test_gpu_mixer as M
from int4_grouped_gemm_router_amd import binding as B

from mixer_ref import BF16_HALF, linear_ref
from ops_ref import U32

pytestmark = pytest.mark.gpu

GUARD = M.GUARD
EDGES = (127, 128, 383, 384)  # the last token of a window of 128 and the first of the next


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"


def bound(o_more=0.0, state_more=0.0):
    """What linear_bound gives, from chunks of 32 tokens and with more for either: a term of the state passes, per chunk, a
    sum of up to 32 terms, a decay (of 4 u: the exponential's ulp, its argument's sums) and a step of the exponent in front
    of the state (2 u, as it stays within 4), and per window (of two chunks at least) a product and a sum, 2 u each: 42 a
    chunk. o adds a sum over dk and over 32 tokens, and with operands of bf16 one rounding of 2^-8 for each product."""
    def f(dk, length, chunked):
        steps = (length + 31) // 32 * 42 + 20 if chunked else 4 * length + 10
        state = steps * U32 + state_more
        return state + o_more + (dk + 40) * U32 + (1.01 * BF16_HALF if chunked else 0.0), state
    return f


def of_sums(largest):
    """Relative error of a decay within a chunk that is 2^(the difference of two sums of up to `largest`), which o's products
    take: each sum is rounded six times, by 2^-24 of it at most (and ln 2 is less than 1). A state's weights are sums from
    their own tokens on, whose error x 2^-24 shrinks with e^-x, and need no such term."""
    return 12 * largest * U32


@pytest.fixture
def case(monkeypatch):
    """linear attention against 64 bits, as the cases of one window are."""
    def run(*a, o_more=0.0, state_more=0.0, **kw):
        monkeypatch.setattr(M, "linear_bound", bound(o_more, state_more))
        M._linear_case(*a, **kw)
    return run


def _windows(plan, n, T):
    """A workspace of a call, which has several windows."""
    ws = B.linear_attention_workspace(plan, n, T)
    assert ws is not None, "one window"
    return ws.fill_(GUARD)


# ------------------------------------------------------------------ linear attention over several windows

@pytest.mark.parametrize("value", [-math.inf, -1e30, -500.0, -90.0])
def test_windows_forget_at_strong_decays(case, value):
    """Strong decays before, at and behind a window's end, and over a whole window."""
    def cut(g):
        g = g.clone()
        for t, h in zip(EDGES, (0, 1, 1, 0)):
            g[t, h] = value
        g[639:642] = value
        g[768:896, 1] = value
        return g
    # (a chunk's sums are limited at 288 a token, 32 of them at most)
    case([30, 1000, 100], Hv=2, decay=cut, o_more=of_sums(288 * 32))
    case([30, 1000, 100], Hk=1, Hv=1, dk=128, dv=40, decay=cut_one(value), scale=-0.7, o_more=of_sums(288 * 3))


def cut_one(value):
    def cut(g):
        g = g.clone()
        for t in (*EDGES, 640, 1100):
            g[t] = value
        return g
    return cut


def test_windows_growth(case):
    """Positive log decays that make e^20 of a state over the windows, and falls that undo them: the windows' sums, of up to
    30 / ln 2 = 44, are rounded once for each of 32 chunks, whose own, of up to 5, are rounded six times."""
    more = 32 * (44 + 6 * 5) * U32
    steady = lambda g: torch.full_like(g, 0.02)  # noqa: E731
    case([1000], Hv=2, decay=steady, o_more=more, state_more=more)
    waves = lambda g: torch.where(torch.arange(len(g))[:, None] // 200 % 2 == 0, 0.1, -0.1).expand_as(g).contiguous()  # noqa: E731
    case([5, 995, 40], Hv=2, decay=waves, o_more=more, state_more=more)


@pytest.mark.parametrize("more", [dict(scale=-1.25), dict(per_token=False, scale=2.0), dict(behind=70, pad=8),
                                  dict(strong=0.3, scale=-0.5, o_more=of_sums(288 * 32))], ids=str)
def test_windows_scales(case, more):
    case([640, 0, 300], Hv=2, **more)


def test_windows_scale_of_zero():
    """Outputs are zeros (of which a relative error says nothing), states those of any other scale, bit for bit."""
    lengths, H, D = [640, 0, 300], 2, 64
    T, n = sum(lengths), len(lengths)
    q, k, v, g = (t.cuda() for t in M._linear_inputs(T, H, H, D, D, True, 3 * T + D))
    pool = torch.randn((n + 2, H, D, D), generator=torch.Generator().manual_seed(5)).cuda()
    cu, states = torch.tensor([0, 640, 640, T], dtype=torch.int32, device="cuda"), []
    for scale in (0.0, 1.0):
        plan = B.linear_attention(H, H, D, D, scale=scale)
        o, S = torch.full_like(v, 5.0), torch.empty((n, H, D, D), device="cuda")
        B.moe_linear_attention(plan, q, k, v, g, o, cu, T, state_in=pool, state_out=S, ws=_windows(plan, n, T))
        assert scale or (o == 0).all()
        states.append(S)
    assert torch.equal(*states) and torch.equal(states[0][1], pool[1])


@pytest.mark.parametrize("c", [dict(lengths=[700, 0, 300], Hk=1, Hv=2, dk=256, dv=256, inplace=True, slots=[4, 1, 0]),
                               dict(lengths=[1100, 30], Hk=1, Hv=1, dk=200, dv=72, inplace=True, slots=[3, 0]),
                               dict(lengths=[64, 900], Hk=1, Hv=1, dk=136, dv=8, slots=[3, 3]),
                               dict(lengths=[600, 700, 1, 64, 0, 9, 8, 100, 3], Hk=1, Hv=1, dk=248, dv=64, inplace=True)], ids=str)
def test_windows_of_wide_heads(case, c):
    """States of more than 128 rows that go over several windows."""
    case(**c)


def _clean(T, H, D, seed, cu):
    q, k, v, g = M._linear_inputs(T, H, H, D, D, True, seed)
    g = g * 0.02  # (decays weak enough for a state to reach the end of its sequence)
    n = len(cu) - 1
    return (q, k, v, g), B.linear_attention(H, H, D, D), torch.tensor(cu, dtype=torch.int32, device="cuda"), n


def _run(plan, cu, n, q, k, v, g):
    T, H, D = v.shape
    o, S = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((n, H, D, D), device="cuda")
    B.moe_linear_attention(plan, q.cuda(), k.cuda(), v.cuda(), g.cuda(), o, cu, T, state_out=S, ws=_windows(plan, n, T))
    return o.cpu(), S.cpu()


@pytest.mark.parametrize("at", EDGES)
def test_windows_nan_decay_reaches_the_rest_of_its_sequence_only(at):
    T, H, D, offsets = 1130, 2, 64, [0, 30, 1030, 1130]
    inputs, plan, cu, n = _clean(T, H, D, 3, offsets)
    o0, S0 = _run(plan, cu, n, *inputs)
    q, k, v, g = inputs
    g = g.clone()
    g[at, 0] = math.nan
    o, S = _run(plan, cu, n, q, k, v, g)
    same = torch.ones((T, H), dtype=torch.bool)
    same[at:1030, 0] = False
    assert torch.equal(o[same], o0[same])
    assert o[~same].isnan().all() and S[1, 0].isnan().all()
    assert torch.equal(S[[0, 2]], S0[[0, 2]]) and torch.equal(S[1, 1], S0[1, 1])


@pytest.mark.parametrize("D,H,at,value", [(64, 2, 383, math.nan), (64, 2, 384, math.inf), (128, 1, 128, -math.inf), (128, 2, 127, math.nan),
                                          (256, 1, 383, math.inf), (40, 1, 384, math.nan)])
def test_windows_not_finite_values_reach_no_earlier_token(D, H, at, value):
    """A NaN or infinity in one token's query, key or value next to a window's end: that token and, but for the query, the
    later ones of its sequence, over all the windows that are left of it (a value: in its column)."""
    T, offsets = 1130, [0, 30, 1030, 1130]
    inputs, plan, cu, n = _clean(T, H, D, 17, offsets)
    want, weight, _, _ = linear_ref(*inputs, torch.zeros((n, H, D, D)), offsets, D ** -0.5)
    ro, _ = bound()(D, 1000, True)
    o0, S0 = _run(plan, cu, n, *inputs)
    for which in range(3):
        bad = [t.clone() for t in inputs]
        bad[which][at, 0, 5] = value
        o, S = _run(plan, cu, n, *bad)
        same = torch.ones((T, H, D), dtype=torch.bool)
        if which == 0:
            same[at, 0] = False
        elif which == 1:
            same[at:1030, 0] = False
        else:
            same[at:1030, 0, 5] = False
        M._close(o[same], want[same], ro * weight[same], torch.bfloat16, f"o beside operand {which}")
        assert not o[~same].isfinite().any(), which
        assert torch.equal(o[:, 1:], o0[:, 1:]) and torch.equal(o[1030:], o0[1030:]) and torch.equal(o[:30], o0[:30])
        assert torch.equal(S[[0, 2]], S0[[0, 2]]) and torch.equal(S[1, 1:], S0[1, 1:])
        if which == 0:
            assert torch.equal(S, S0)
        elif which == 2:
            assert not S[1, 0, :, 5].isfinite().any() and torch.equal(S[1, 0, :, :5], S0[1, 0, :, :5])


def test_windows_offsets_out_of_order_stay_in_range():
    """Offsets that decrease or leave 0..T, in calls of several windows and of more sequences than a wave holds: nothing
    outside the outputs, the states and the workspace is touched."""
    T, H, D = 1200, 1, 32
    q, k, v, g = (t.cuda() for t in M._linear_inputs(T, H, H, D, D, True, 8))
    plan = B.linear_attention(H, H, D, D)
    gen = torch.Generator().manual_seed(6)
    many = torch.randint(-100, 3000, (90,), generator=gen).tolist()
    for cu in ([0, 700, 5000], [-7, 900, 1 << 30], [0, 800, 300, 2000000000], [1100, 10, -5], many, sorted(many), sorted(many)[::-1]):
        n = len(cu) - 1
        o = torch.full((T + 4, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
        S = torch.full((n + 1, H, D, D), 3.0, device="cuda")
        size = _windows(plan, n, T).numel()
        ws = torch.full((size + 4096,), GUARD, dtype=torch.uint8, device="cuda")
        B.moe_linear_attention(plan, q, k, v, g, o, torch.tensor(cu, dtype=torch.int32, device="cuda"), T, state_out=S[:n], ws=ws[:size])
        torch.cuda.synchronize()
        assert (o[T:] == 3.0).all() and (S[n] == 3.0).all() and (ws[size:] == GUARD).all()


def test_as_many_windows_as_there_can_be(case):
    """70000 tokens of one head: 512 windows, several of them within a sequence, others with many sequences."""
    case([40000, 0, 3, 200] + [9] * 40 + [300] * 50 + [70000 - 40000 - 203 - 360 - 15000], Hk=1, Hv=1, dk=16, dv=8)


def test_as_many_sequences_as_there_can_be():
    """65536 sequences, single tokens but for three: by the step, and in one call with the others."""
    n, H, D, scale = 65536, 1, 8, 0.5
    g = torch.Generator().manual_seed(3)
    lengths = torch.ones(n, dtype=torch.int64)
    lengths[0], lengths[30000], lengths[n - 1] = 40, 600, 9
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    T = int(cu[-1])
    q, k, v = ((torch.randn((T, H, D), generator=g) / 2).bfloat16() for _ in range(3))
    decay = -torch.rand((T, H), generator=g) * 0.1
    pool = torch.randn((n, H, D, D), generator=g)
    plan = B.linear_attention(H, H, D, D, scale=scale)

    def single(at, S, o):
        """Those tokens as sequences of their own, whose states are those of `pool`."""
        S0 = pool[S].double()
        want = torch.exp(decay[at].double())[..., None, None] * S0 + k[at].double()[..., None] * v[at].double()[:, :, None, :]
        size = torch.exp(decay[at].double())[..., None, None] * S0.abs() + (k[at].double()[..., None] * v[at].double()[:, :, None, :]).abs()
        y = scale * (q[at].double()[..., None] * want).sum(2)
        weight = scale * (q[at].double()[..., None].abs() * size).sum(2)
        ro, rs = bound()(D, 1, False)
        M._close(o, y, ro * weight, torch.bfloat16, "o")
        return want, rs * size + 1e-37
    o, S = torch.empty((n, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((n, H, D, D), device="cuda")
    B.moe_linear_attention_step(plan, q[:n].cuda(), k[:n].cuda(), v[:n].cuda(), decay[:n].cuda(), o, n, state_in=pool.cuda(), state_out=S)
    want, err = single(slice(0, n), slice(0, n), o)
    assert ((S.cpu().double() - want).abs() <= err).all()

    o, S = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda"), pool.cuda()
    B.moe_linear_attention(plan, q.cuda(), k.cuda(), v.cuda(), decay.cuda(), o, cu.to(torch.int32).cuda(), T, state_in=S, state_out=S,
                           ws=_windows(plan, n, T))
    one = lengths == 1
    at = cu[:-1][one]
    want, err = single(at, one, o.cpu()[at])
    assert ((S.cpu().double()[one] - want).abs() <= err).all()
    for i in (0, 30000, n - 1):
        part = slice(int(cu[i]), int(cu[i + 1]))
        L = int(lengths[i])
        y, weight, states, sums = linear_ref(q[part], k[part], v[part], decay[part], pool[i:i + 1], [0, L], scale)
        ro, rs = bound()(D, L, True)
        M._close(o[part], y, ro * weight, torch.bfloat16, f"o of sequence {i}")
        assert ((S[i].cpu().double() - states[0]).abs() <= rs * sums[0] + 1e-37).all()


@pytest.mark.parametrize("n", [2, 9])
def test_linear_empty_sequences_copy_their_states(n):
    """The state of a sequence without tokens arrives as it is, large and small values, infinities and NaN among them."""
    H, D = 2, 64
    plan = B.linear_attention(H, H, D, D)
    pool = torch.randn((n, H, D, D), generator=torch.Generator().manual_seed(1))
    pool[1, 0, 0, :6] = torch.tensor([1e38, -1e-37, 2.0 ** -126, math.inf, -math.inf, math.nan])
    q = torch.randn((4, H, D), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    cu = torch.tensor([0, 4] + [4] * (n - 1), dtype=torch.int32, device="cuda")
    S, o = torch.full((n, H, D, D), 7.0, device="cuda"), torch.empty_like(q)
    B.moe_linear_attention(plan, q, q, q, torch.zeros((4, H), device="cuda"), o, cu, 4, state_in=pool.cuda(), state_out=S)
    assert torch.equal(S[1:].cpu().nan_to_num(nan=5.0), pool[1:].nan_to_num(nan=5.0)) and S[1, 0, 0, 5].isnan()


# ------------------------------------------------------------------ the norm after a block

@pytest.mark.parametrize("H", [128, 100, 500, 1000, 2048, 2500, 8192, 9000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_norm_infinite_gate_of_a_row(H, dtype):
    """An infinite gate of a row makes it infinite, and so the scale of its 8-bit values, at every width."""
    dt = M.DT[dtype]
    x = (torch.rand((3, H), generator=torch.Generator().manual_seed(H)) + 0.5).to(dt)
    z = torch.tensor([[1.0], [math.inf], [-2.0]]).to(dt)
    for out8, kind in ((B.OUT8_INT8, torch.int8), (B.OUT8_E4M3, torch.float8_e4m3fn)):
        n = B.gated_norm(H, dtype=dt, normalize=False, gate=B.GATE_SILU, gate_per_row=True, out8=out8)
        h, q, s = torch.empty_like(x).cuda(), torch.empty((3, H), dtype=kind, device="cuda"), torch.empty((3, 1), device="cuda")
        B.moe_gated_norm(n, x.cuda(), 3, gate=z.cuda(), h_out=h, q=q, scales=s)
        assert (h[1] == math.inf).all() and h[[0, 2]].isfinite().all()
        assert s[1, 0] == math.inf and s[[0, 2]].isfinite().all(), s
        assert (q[1] == 0).all() if out8 == B.OUT8_INT8 else q[1].float().isnan().all()


# ------------------------------------------------------------------ together

def test_windows_in_graphs_that_share_a_workspace():
    """Two captured blocks of several windows each with one workspace, replayed in turn with eager work between them and
    the workspace overwritten, and on another stream: the same bits as the eager run."""
    ms = [M._Mixer(sum(s), s, seed=i).to_gpu() for i, s in enumerate(([900, 13], [7, 700]))]
    for m in ms:
        assert m.ws[1] is not None, "one window"
    assert ms[0].ws[1].numel() != ms[1].ws[1].numel()     # (windows differ in number)
    want = []
    for m in ms:
        m.run()
        want.append(m.outputs())
        m.check(want[-1])
    big = max((m.ws[1] for m in ms), key=torch.Tensor.numel)
    for m in ms:
        m.ws = (m.ws[0], big, m.ws[2])
    assert ms[0].ws[1].data_ptr() == ms[1].ws[1].data_ptr()
    graphs = []
    for m in ms:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.run()
        graphs.append(g)
    for turn in range(4):
        for m, g, w in zip(ms, graphs, want):
            for t in m.b.values():
                t.fill_(3)
            if turn != 1:
                big.fill_(0xFF if turn else GUARD)        # (0xFF: NaN in every value)
            if turn % 2:
                torch.cuda.synchronize()
            g.replay()
            got = m.outputs()
            assert all(torch.equal(got[n], w[n]) for n in w), turn
            (torch.ones(1000, device="cuda") * 2).sum().item()
    # one behind the other without a wait between them, and eagerly on another stream
    for m in ms:
        for t in m.b.values():
            t.fill_(3)
    graphs[0].replay()
    graphs[1].replay()
    for m, w in zip(ms, want):
        got = m.outputs()
        assert all(torch.equal(got[n], w[n]) for n in w)
        for t in m.b.values():
            t.fill_(3)
    big.fill_(0xFF)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for m in ms:
            m.run()
    for m, w in zip(ms, want):
        got = m.outputs()
        assert all(torch.equal(got[n], w[n]) for n in w)


class _Step(M._Mixer):
    """A block of one token for each of a pool's sequences: the mixer's weights, states in place."""

    def __init__(self, n, pool, slots, positions, seed, tokens):
        super().__init__(n, [1] * n, seed=seed)
        g = torch.Generator().manual_seed(tokens)
        self.x, self.res = (torch.randn((n, self.H), generator=g).bfloat16() for _ in range(2))
        self.decay = -torch.rand((n, self.Hv), generator=g) * 0.2
        self.positions = positions
        self.pool, self.slots = pool, slots

    def run(self):
        whole = B.moe_linear_attention

        def step(plan, q, k, v, decay, o, cu, T, state_out, ws):
            B.moe_linear_attention_step(plan, q, k, v, decay, o, T, state_in=self.pool, slots_in=self.slots, state_out=self.pool,
                                        slots_out=self.slots)
        B.moe_linear_attention = step
        try:
            super().run()
        finally:
            B.moe_linear_attention = whole
        self.b["S"].copy_(self.pool[self.slots.long()])


@pytest.mark.parametrize("lengths", [[40, 3], [900, 13, 1]], ids=str)
def test_mixer_prompt_then_single_tokens(monkeypatch, lengths):
    """A block's prompts, and then single tokens of the same sequences out of the pool that holds their states."""
    monkeypatch.setattr(M, "linear_bound", bound())
    n, D = len(lengths), 64
    prompt = M._Mixer(sum(lengths), lengths, seed=5).to_gpu()
    assert (prompt.ws[1] is not None) == (max(lengths) > 500)
    prompt.run()
    first = prompt.outputs()
    prompt.check(first)
    pool = torch.full((n + 2, prompt.Hv, D, D), 9.0, device="cuda")
    slots = torch.tensor([n + 1 - i for i in range(n)], dtype=torch.int32, device="cuda")
    pool[slots.long()] = prompt.b["S"]
    start = first["S"]
    for i in range(4):
        positions = torch.tensor([L + i for L in lengths], dtype=torch.int32)
        s = _Step(n, pool, slots, positions, 5, 100 + i).to_gpu()
        assert torch.equal(s.w_in, prompt.w_in) and torch.equal(s.w_out, prompt.w_out)
        s.run()
        got = s.outputs()
        monkeypatch.setattr(M, "linear_ref", lambda q, k, v, g, _, cu, scale: linear_ref(q, k, v, g, start, cu, scale))  # noqa: B023
        s.check(got)
        monkeypatch.setattr(M, "linear_ref", linear_ref)
        start = got["S"]
    assert (pool[:2] == 9.0).all()
