"""GPU parity of linear attention with a decay for each head against the float64 oracle's recurrence:
prompts, single tokens and gradients.

Bars, as the 2-norm of the difference over the 2-norm of the result (u = 2^-24, float32's unit
roundoff; v = 2^-9 bounds what a rounding to bfloat16 adds in that norm: errors spread evenly up to
2^-8 of a value's power of two, that is 2^-8 / sqrt(3) of a number 1.4 times smaller than the value):
 - float32: an output is a sum of at most 256 products over a state that was rounded once a chunk
   and once a step in it, sqrt(256) + sqrt(32 + T / 32) roundings at random, and its decays are
   exponentials of sums of up to 100 in base 2, each off by 100 u at most: together under 128 u,
   7.6e-6; the bar is 1e-5.
 - bfloat16 outputs: their own rounding (v), that of the scores and that of the state as an operand,
   each v of their part: 3 v.
 - float32 states of bfloat16 operands: the scaled values are split into bfloat16 terms that leave
   at most 2^-17 of each: 2^-17 + 1e-5 < 2e-5.
 - the log decays' gradient is a sum from the end of T terms r - c that cancel, each off by at most
   1e-5 of its size at random: 1e-5 sqrt(2 T) rms(r), compared with the largest difference / 4."""
import numpy as np
import pytest
import torch

from oracle import block_ops as ref
from parity import case, to_np

pytestmark = pytest.mark.gpu

DEV = "cuda"
V = 2.0 ** -9
F32_BAR, BF16_BAR, STATE_BAR = 1e-5, 3 * V, 2e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def amd(gpu_lib):
    import recurrent_nets_amd
    return recurrent_nets_amd


def _rel(got, want):
    got, want = to_np(got), np.asarray(want)
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.all(np.isfinite(got))
    n = np.linalg.norm(want)
    return float(np.linalg.norm(got - want) / n) if n > 0 else float(np.linalg.norm(got))


class Problem:
    """Inputs on the host and the device, and the oracle's results."""

    def __init__(self, seed, B, T, H, dk, dv, dtype="f32", layout="bthd", state0=True, g_final=False, cu=None, gate=None,
                 per_head=False):
        r = np.random.default_rng(seed)
        dt = DT[dtype]

        def rand(*shape):
            return torch.from_numpy(r.standard_normal(shape).astype(np.float32))
        self.n = B if cu is None else len(cu) - 1
        self.cu = cu
        self.scale = float(np.float32(dk ** -0.5))
        self.bar = BF16_BAR if dtype == "bf16" else F32_BAR
        self.go = rand(B, T, H, dv).to(dt).to(DEV)
        if layout == "slices":
            assert dk == dv
            P = rand(B, T, 4, H * dk).to(dt).to(DEV)
            self.q, self.k, self.v = (P[:, :, i].view(B, T, H, dk) for i in range(3))
        elif layout == "bhtd":
            self.q, self.k, self.v = (rand(B, H, T, d).to(dt).to(DEV).transpose(1, 2) for d in (dk, dk, dv))
            self.go = rand(B, H, T, dv).to(dt).to(DEV).transpose(1, 2)
        else:
            self.q, self.k, self.v = (rand(B, T, H, d).to(dt).to(DEV) for d in (dk, dk, dv))
        if per_head:
            g = -np.exp(r.uniform(-6, 0, H))
        else:
            g = -np.logaddexp(0.0, -(r.standard_normal((B, T, H)) + np.linspace(0.0, 5.0, H)))
        g = g.astype(np.float32)
        if gate is not None:
            g = gate(g, r).astype(np.float32)
        self.g = torch.from_numpy(g).to(DEV)
        self.s0 = rand(self.n, H, dk, dv).to(DEV) if state0 else None
        self.gf = rand(self.n, H, dk, dv).to(DEV) if g_final else None
        self.shape = (B, T, H, dk, dv)

    def _items(self):
        B, T, H, _, _ = self.shape
        spans = [(b, 0, T) for b in range(B)] if self.cu is None else [(0, a, b) for a, b in zip(self.cu, self.cu[1:])]
        g = to_np(self.g)
        g = np.broadcast_to(g, (B, T, H)) if g.ndim == 1 else g
        q, k, v, go = (to_np(x) for x in (self.q, self.k, self.v, self.go))
        s0, gf = (None if x is None else to_np(x) for x in (self.s0, self.gf))
        for s, (b, a, e) in enumerate(spans):
            for h in range(H):
                at = (b, slice(a, e), h)
                yield s, h, at, q[at], k[at], v[at], g[at], go[at], None if s0 is None else s0[s, h], None if gf is None else gf[s, h]

    def forward(self):
        B, T, H, dk, dv = self.shape
        o, S = np.zeros((B, T, H, dv)), np.zeros((self.n, H, dk, dv))
        for s, h, at, q, k, v, g, _, s0, _ in self._items():
            o[at], states = ref.linear_attention(q, k, v, g, s0, self.scale)
            S[s, h] = states[-1]
        return o, S

    def backward(self):
        B, T, H, dk, dv = self.shape
        dq, dk_, dv_, dg = np.zeros((B, T, H, dk)), np.zeros((B, T, H, dk)), np.zeros((B, T, H, dv)), np.zeros((B, T, H))
        ds = np.zeros((self.n, H, dk, dv))
        for s, h, at, q, k, v, g, go, s0, gf in self._items():
            dq[at], dk_[at], dv_[at], dg[at], ds[s, h] = ref.linear_attention_backward(q, k, v, g, go, s0, gf, self.scale)
        return dq, dk_, dv_, dg, ds

    def check_forward(self, amd, **kw):
        o, S = amd.linear_attention_forward(self.q, self.k, self.v, self.g, self.s0, scale=self.scale, want_final_state=True,
                                            cu_seqlens=self.cu, **kw)
        torch.cuda.synchronize()
        wo, wS = self.forward()
        assert o.dtype == self.q.dtype
        eo, eS = _rel(o, wo), _rel(S, wS)
        assert eo < self.bar and eS < STATE_BAR, (eo, eS)
        return o, S

    def check_backward(self, amd, **kw):
        B, T, H, dk, dv = self.shape
        dq, dk_, dv_, dg, ds = amd.linear_attention_backward(self.q, self.k, self.v, self.g, self.go, self.s0, self.gf,
                                                             scale=self.scale, want_dstate0=True, cu_seqlens=self.cu, **kw)
        torch.cuda.synchronize()
        w = self.backward()
        errs = [_rel(a, b) for a, b in zip((dq, dk_, dv_), w)]
        assert max(errs) < self.bar, errs
        assert _rel(ds, w[4]) < STATE_BAR
        if dg is not None:
            r = np.einsum("bthd,bthd->bth", to_np(self.q), w[0])
            size = np.sqrt(np.mean(r * r)) + np.sqrt(np.mean(w[3] ** 2))
            off = np.max(np.abs(to_np(dg) - w[3]), initial=0.0)
            assert off <= 4 * 1e-5 * np.sqrt(2 * T) * size, (off, size)
        return dq, dk_, dv_, dg, ds


# ---- prompts ------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 77, 129, 300])
def test_lengths(amd, T, dtype):
    p = Problem(100 + T, 2, T, 3, 64, 64, dtype, g_final=True)
    case(f"linear attention T={T} {dtype}")
    p.check_forward(amd)
    p.check_backward(amd)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(8, 8), (16, 40), (40, 16), (32, 256), (256, 32), (64, 128), (128, 64), (96, 128), (200, 72),
                                   (256, 256), (128, 256)])
def test_widths(amd, dk, dv, dtype):
    p = Problem(dk * 300 + dv, 1, 70, 2, dk, dv, dtype, g_final=True)
    case(f"linear attention widths {dk}, {dv} {dtype}")
    p.check_forward(amd)
    p.check_backward(amd)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bhtd", "slices"])
def test_layouts(amd, layout, dtype):
    p = Problem(7, 2, 75, 3, 48, 48, dtype, layout=layout, state0=False)
    case(f"linear attention layout {layout} {dtype}")
    o, _ = p.check_forward(amd)
    dq, dk, dv, _, _ = p.check_backward(amd)
    # outputs in place: the slices of one gradient, a transposed output
    B, T, H, d, _ = p.shape
    dP = torch.full((B, T, 4, H * d), 7.0, dtype=p.q.dtype, device=DEV)
    views = [dP[:, :, i].view(B, T, H, d) for i in range(3)]
    amd.linear_attention_backward(p.q, p.k, p.v, p.g, p.go, scale=p.scale, dq=views[0], dk=views[1], dv=views[2])
    ot = torch.empty((B, H, T, d), dtype=p.q.dtype, device=DEV)
    amd.linear_attention_forward(p.q, p.k, p.v, p.g, scale=p.scale, out=ot.transpose(1, 2))
    torch.cuda.synchronize()
    for got, want in zip(views + [ot.transpose(1, 2)], (dq, dk, dv, o)):
        assert torch.equal(got, want)
    assert bool((dP[:, :, 3] == 7.0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_time_segments(amd, dtype):
    """One long sequence: the time axis runs in segments that are joined."""
    p = Problem(11, 1, 1000, 2, 64, 32, dtype, g_final=True)
    assert amd.linear_attention.linear_attention_workspace_bytes(1, 1000, 2, 64, 32) > 0
    case(f"linear attention in segments {dtype}")
    p.check_forward(amd)
    p.check_backward(amd)


def test_many_heads_in_one_segment(amd):
    p = Problem(12, 80, 67, 8, 16, 16, "bf16", state0=False)
    assert amd.linear_attention.linear_attention_workspace_bytes(80, 67, 8, 16, 16) == 0
    case("linear attention, 640 heads")
    p.check_forward(amd)
    p.check_backward(amd)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decay_per_head(amd, dtype):
    p = Problem(13, 2, 200, 4, 32, 32, dtype, per_head=True, g_final=True)
    case(f"linear attention, fixed decays {dtype}")
    p.check_forward(amd)
    _, _, _, dg, _ = p.check_backward(amd)
    assert dg is None


def _starts(g, r):
    g[:, 0] = -np.inf
    g[:, 5:9] = -np.inf
    g[:, 40] = -104.0
    g[:, 64] = -1e30
    return g


def _all_resets(g, r):
    return np.full_like(g, -np.inf)


def _no_decay(g, r):
    return np.zeros_like(g)


def _strong(g, r):
    return -r.uniform(0, 60, g.shape)


def _growing(g, r):
    return r.uniform(-0.2, 0.1, g.shape)


def _long(g, r):
    return -10.0 ** r.uniform(-5, -2.5, g.shape[-1:]) * np.ones(g.shape)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_memories(amd, dtype):
    """Decays that remember thousands of steps, over as many: small exponents add up exactly."""
    p = Problem(16, 1, 3000, 6, 32, 32, dtype, gate=_long, g_final=True)
    case(f"linear attention, long memories {dtype}")
    p.check_forward(amd)
    p.check_backward(amd)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [_starts, _all_resets, _no_decay, _strong, _growing])
def test_decays(amd, gate, dtype):
    p = Problem(17, 2, 97, 2, 32, 64, dtype, gate=gate, g_final=True)
    case(f"linear attention decays {gate.__name__} {dtype}")
    p.check_forward(amd)
    _, _, _, dg, ds = p.check_backward(amd)
    dead = torch.from_numpy(to_np(p.g) <= -104.0).to(DEV)
    assert bool((dg[dead] == 0).all())
    if gate is _starts:
        assert bool((ds == 0).all())


def test_first_step_without_a_state_has_no_decay_gradient(amd):
    p = Problem(18, 3, 1, 2, 16, 16, "f32", state0=False)
    case("linear attention, one step, no state")
    _, _, _, dg, _ = p.check_backward(amd)
    assert bool((dg == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 5, 5, 38, 100], [0, 0, 0, 64], [0, 300, 301, 640, 640]])
def test_packed(amd, cu, dtype):
    p = Problem(19 + len(cu) + cu[-1], 1, cu[-1], 2, 32, 48, dtype, cu=cu, g_final=True)
    case(f"linear attention packed {cu} {dtype}")
    _, S = p.check_forward(amd)
    p.check_backward(amd)
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        if a == b:
            assert torch.equal(S[s], p.s0[s])


def test_packed_many(amd):
    """More sequences than segments, offsets on the device."""
    rng = np.random.default_rng(3)
    cu = [0] + np.cumsum(rng.integers(0, 9, 300)).tolist()
    p = Problem(23, 1, cu[-1], 1, 16, 16, "f32", cu=cu, state0=False)
    case("linear attention, 300 packed sequences")
    p.check_forward(amd)
    p.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o, S = amd.linear_attention_forward(p.q, p.k, p.v, p.g, scale=p.scale, want_final_state=True, cu_seqlens=p.cu)
    p.cu = cu
    torch.cuda.synchronize()
    wo, wS = p.forward()
    assert _rel(o, wo) < F32_BAR and _rel(S, wS) < STATE_BAR


def test_no_steps(amd):
    s0 = torch.randn(2, 3, 16, 8, device=DEV)
    q, v = torch.empty(2, 0, 3, 16, device=DEV), torch.empty(2, 0, 3, 8, device=DEV)
    g = torch.empty(2, 0, 3, device=DEV)
    case("linear attention, no steps")
    o, S = amd.linear_attention_forward(q, q, v, g, s0, want_final_state=True)
    dq, dk, dv, dg, ds = amd.linear_attention_backward(q, q, v, g, v, s0, g_final=s0, want_dstate0=True)
    torch.cuda.synchronize()
    assert o.shape == v.shape and torch.equal(S, s0) and dg.shape == g.shape and torch.equal(ds, s0)


@pytest.mark.parametrize("T,cut", [(150, 61), (1500, 700)])
def test_continued_prompt_in_place(amd, T, cut):
    """A prompt in two parts, the state passed on in its own buffer, also in segments of time."""
    p = Problem(29, 2, T, 2, 32, 32, "f32")
    case("linear attention continued")
    whole, S = p.check_forward(amd)
    state = p.s0.clone()
    parts = []
    for sl in (slice(0, cut), slice(cut, T)):
        o, _ = amd.linear_attention_forward(p.q[:, sl], p.k[:, sl], p.v[:, sl], p.g[:, sl].contiguous(), state, scale=p.scale,
                                            final_state=state)
        parts.append(o)
    torch.cuda.synchronize()
    assert _rel(torch.cat(parts, 1), to_np(whole)) < 2 * F32_BAR and _rel(state, to_np(S)) < 2 * F32_BAR


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["k", "v", "g"])
def test_what_is_not_finite_stays_in_the_future(amd, where, bad, dtype):
    """A step's outputs depend on the steps up to it only."""
    p = Problem(31, 1, 90, 2, 32, 40, dtype)
    clean, _ = amd.linear_attention_forward(p.q, p.k, p.v, p.g, p.s0, scale=p.scale)
    at = 45
    if where == "g":
        p.g[:, at] = bad
    else:
        getattr(p, where)[:, at, :, 3] = bad
    case(f"linear attention with {bad} in {where} {dtype}")
    o, S = amd.linear_attention_forward(p.q, p.k, p.v, p.g, p.s0, scale=p.scale, want_final_state=True)
    torch.cuda.synchronize()
    assert bool(o[:, :at].isfinite().all())
    assert _rel(o[:, :at], to_np(clean[:, :at])) < p.bar
    assert not bool(o[:, at].isfinite().all()) and not bool(S.isfinite().all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where,name", [("k", "dq"), ("v", "dq"), ("q", "dk"), ("go", "dk"), ("go", "dv"), ("q", "dv")])
def test_gradients_keep_to_their_side_too(amd, where, name, dtype):
    """dq takes earlier keys and values; dk and dv take later queries and gradients."""
    p = Problem(37, 1, 90, 1, 32, 32, dtype)
    clean = dict(zip(("dq", "dk", "dv"), amd.linear_attention_backward(p.q, p.k, p.v, p.g, p.go, p.s0, scale=p.scale)))
    getattr(p, where)[:, 45, :, 3] = float("nan")
    case(f"linear attention gradients with NaN in {where} {dtype}")
    got = dict(zip(("dq", "dk", "dv"), amd.linear_attention_backward(p.q, p.k, p.v, p.g, p.go, p.s0, scale=p.scale)))
    torch.cuda.synchronize()
    side = slice(0, 45) if name == "dq" else slice(46, 90)
    assert bool(got[name][:, side].isfinite().all())
    assert _rel(got[name][:, side], to_np(clean[name][:, side])) < p.bar


def test_steps_after_a_reset_do_not_see_what_was_before(amd):
    """Whatever it was: NaN in an earlier document stays there."""
    p = Problem(39, 1, 100, 2, 32, 32, "bf16", gate=_starts)
    clean, S = amd.linear_attention_forward(p.q, p.k, p.v, p.g, p.s0, scale=p.scale, want_final_state=True)
    p.k[:, 50, :, 3] = float("nan")
    p.v[:, 51, :, 3] = float("inf")
    case("linear attention, NaN before a reset")
    o, S2 = amd.linear_attention_forward(p.q, p.k, p.v, p.g, p.s0, scale=p.scale, want_final_state=True)
    torch.cuda.synchronize()
    assert torch.equal(o[:, 64:], clean[:, 64:]) and torch.equal(S, S2)
    assert torch.equal(o[:, :50], clean[:, :50])


# ---- single tokens --------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 8, 8), (3, 2, 64, 64), (2, 3, 40, 72), (5, 2, 256, 128), (4, 1, 128, 256)])
def test_step(amd, B, H, dk, dv, dtype):
    p = Problem(41 + dk + dv, B, 1, H, dk, dv, dtype)
    wo, wS = p.forward()
    pool = torch.randn(B + 4, H, dk, dv, device=DEV)
    before = pool.clone()
    slots = torch.randperm(B + 4, device=DEV)[:B].to(torch.int32)
    pool[slots.long()] = p.s0
    case(f"linear attention step B={B} H={H} {dk}, {dv} {dtype}")
    o = amd.linear_attention_step(p.q[:, 0], p.k[:, 0], p.v[:, 0], p.g[:, 0].contiguous(), pool, slots=slots, scale=p.scale)
    torch.cuda.synchronize()
    # outputs are rounded once; the state is float32 arithmetic on exact operands
    assert _rel(o, wo[:, 0]) < (V if dtype == "bf16" else F32_BAR)
    assert _rel(pool[slots.long()], wS) < F32_BAR
    rest = [i for i in range(B + 4) if i not in slots.tolist()]
    assert torch.equal(pool[rest], before[rest])


def test_step_slots_outside_the_pool(amd):
    p = Problem(43, 4, 1, 2, 32, 40, "f32")
    pool = p.s0.clone()
    slots = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device=DEV)
    case("linear attention step with slots outside the pool")
    o = amd.linear_attention_step(p.q[:, 0], p.k[:, 0], p.v[:, 0], p.g[:, 0].contiguous(), pool, slots=slots, scale=p.scale)
    torch.cuda.synchronize()
    assert bool((o[1] == 0).all()) and bool((o[2] == 0).all()) and not bool((o[0] == 0).all())
    assert torch.equal(pool[1], p.s0[1]) and torch.equal(pool[3], p.s0[3])
    assert not torch.equal(pool[2], p.s0[2])


def test_steps_follow_the_prompt(amd):
    """Decoding token by token from a prompt's final state is the longer prompt."""
    p = Problem(47, 2, 50, 2, 64, 32, "bf16", layout="bhtd", state0=False, per_head=True)
    case("linear attention steps after a prompt")
    _, S = amd.linear_attention_forward(p.q[:, :40], p.k[:, :40], p.v[:, :40], p.g, scale=p.scale, want_final_state=True)
    outs = [amd.linear_attention_step(p.q[:, t], p.k[:, t], p.v[:, t], p.g, S, scale=p.scale) for t in range(40, 50)]
    torch.cuda.synchronize()
    wo, wS = p.forward()
    assert _rel(torch.stack(outs, 1), wo[:, 40:]) < BF16_BAR
    assert _rel(S, wS) < STATE_BAR


# ---- how it runs ------------------------------------------------------------------------------------
def test_same_bits_on_every_run_and_stream(amd):
    p = Problem(53, 2, 400, 2, 64, 64, "bf16", g_final=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    case("linear attention on a side stream")
    runs = []
    for stream in (None, s, None):
        with torch.cuda.stream(s if stream is not None else torch.cuda.current_stream()):
            o = amd.linear_attention_forward(p.q, p.k, p.v, p.g, p.s0, scale=p.scale, want_final_state=True, stream=stream)
            b = amd.linear_attention_backward(p.q, p.k, p.v, p.g, p.go, p.s0, p.gf, scale=p.scale, want_dstate0=True, stream=stream)
        torch.cuda.synchronize()
        runs.append(o + b)
    for other in runs[1:]:
        for x, y in zip(runs[0], other):
            assert torch.equal(x, y)


def test_graph_replays(amd):
    p = Problem(59, 2, 300, 2, 32, 32, "bf16")
    B, T, H, dk, dv = p.shape
    o, S = amd.linear_attention_forward(p.q, p.k, p.v, p.g, p.s0, want_final_state=True)
    outs = amd.linear_attention_backward(p.q, p.k, p.v, p.g, p.go, p.s0)
    pool = p.s0.clone()
    tok = [x[:, 0] for x in (p.q, p.k, p.v)]
    g0 = p.g[:, 0].contiguous()
    os_ = amd.linear_attention_step(*tok, g0, pool.clone())
    la = amd.linear_attention
    wf = torch.empty(max(1, la.linear_attention_workspace_bytes(B, T, H, dk, dv)), dtype=torch.uint8, device=DEV)
    wb = torch.empty(la.linear_attention_backward_workspace_bytes(B, T, H, dk, dv), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    case("linear attention in a graph")
    with torch.cuda.graph(graph):
        amd.linear_attention_forward(p.q, p.k, p.v, p.g, p.s0, out=o, final_state=S, workspace=wf)
        amd.linear_attention_backward(p.q, p.k, p.v, p.g, p.go, p.s0, dq=outs[0], dk=outs[1], dv=outs[2],
                                      dlog_decay=outs[3], workspace=wb)
        amd.linear_attention_step(*tok, g0, pool, out=os_)
    want_pool = p.s0.clone()
    for i in range(3):
        p.v.mul_(1.0 + 0.5 * i)
        graph.replay()
        torch.cuda.synchronize()
        want = amd.linear_attention_forward(p.q, p.k, p.v, p.g, p.s0, want_final_state=True)
        want += amd.linear_attention_backward(p.q, p.k, p.v, p.g, p.go, p.s0)[:4]
        want += (amd.linear_attention_step(*tok, g0, want_pool), want_pool)
        torch.cuda.synchronize()
        for got, w in zip((o, S) + tuple(outs[:4]) + (os_, pool), want):
            assert torch.equal(got, w)
