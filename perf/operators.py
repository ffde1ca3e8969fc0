"""The measured cases of layer norm and of linear attention with a decay for each head.

Layer norm in both directions, as it stands in front of an input projection; linear attention
as prompts (chunked, whole or packed), single tokens over a pool of states, and training. Sizes
follow this repository's workloads: batch 128 x 2048 steps x 1024 features, 16 x 4096 x 1024,
4 x 16384 x 2048, 8 x 1024 x 256, and decoding at batch 128.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_EPS = 1e-5
_lib = None


# ---- cases --------------------------------------------------------------------------------------
def _norm(name, op, rows, width, dtype, out):
    c = {"op": op, "rows": rows, "width": width, "dtype": dtype, "out": out}
    return {"name": name, **c} if name else c


def _attn(name, op, B, T, H, dk, dv, dtype, gate="token", layout="bthd", state0=False, packed=0, resets=False):
    c = {"op": op, "B": B, "T": T, "H": H, "dk": dk, "dv": dv, "dtype": dtype, "gate": gate, "layout": layout,
         "state0": state0, "packed": packed, "resets": resets}
    return {"name": name, **c} if name else c


def _step(name, B, H, dk, dv, dtype, slots):
    c = {"op": "step", "B": B, "H": H, "dk": dk, "dv": dv, "dtype": dtype, "slots": slots}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the norm in front of one decoded token of 128 sequences: latency
        _norm("norm decode 128x1024", "norm_forward", 128, 1024, "bf16", "bf16"),
        # the norm of a whole layer's tokens, float32 residual stream into the bf16 projection
        _norm("norm layer 262144x1024", "norm_forward", 128 * 2048, 1024, "f32", "bf16"),
        # its backward in bf16, for the batch of 16 x 4096 steps
        _norm("norm grad 65536x1024", "norm_backward", 16 * 4096, 1024, "bf16", "bf16"),
        # backward of a small ragged batch at an odd width
        _norm("norm grad ragged 777x250", "norm_backward", 777, 250, "f32", "f32"),
        # one token for one user: latency
        _step("step b1", 1, 4, 64, 64, "bf16", 8),
        # one token for 128 users, states in a pool of slots
        _step("step b128", 128, 8, 128, 128, "bf16", 192),
        # a short prompt whose q, k, v are slices of one float32 projection
        _attn("prompt short slices", "prompt", 3, 77, 4, 64, 64, "f32", layout="slices", state0=True),
        # ragged prompts packed end to end, documents of different lengths, narrower keys than values
        _attn("prompt packed 24", "prompt", 1, 6001, 8, 64, 128, "bf16", packed=24, state0=True),
        # few long sequences: the time axis has to be split
        _attn("prompt long 4x16384", "prompt", 4, 16384, 16, 128, 128, "bf16", gate="head"),
        # a full batch of prompts
        _attn("prompt layer 128x2048", "prompt", 128, 2048, 8, 128, 128, "bf16", state0=True),
        # training on the float32 projection's slices, documents separated by resets
        _attn("train slices 8x1024", "train", 8, 1024, 4, 64, 64, "f32", layout="slices", resets=True),
        # training in bf16, the batch of 16 x 4096 steps
        _attn("train 16x4096", "train", 16, 4096, 8, 128, 128, "bf16", state0=True),
    ]


def _log(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - 1 if n == 3 * 1024 else n


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "step", "prompt", "prompt", "train", "train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        width = _log(rng, 16, 4096)
        rows = _log(rng, 1, min(300000, (1 << 27) // width))
        return _norm(None, op, rows, width, dtype, rng.choice(["bf16", "f32"]) if op == "norm_forward" else dtype)
    dk, dv = (8 * _log(rng, 2, 32) for _ in range(2))
    H = _log(rng, 1, 16)
    H -= 3 * 1024 in (H * dk, H * dv)
    if op == "step":
        B = _log(rng, 1, max(1, min(512, (1 << 24) // (H * dk * dv))))
        return _step(None, B, H, dk, dv, dtype, B + rng.randrange(0, 64))
    T = _log(rng, 1, 16384 if op == "prompt" else 4096)
    most = (1 << 26) if op == "prompt" else (1 << 24)  # values of one operand
    B = _log(rng, 1, max(1, min(128, most // (T * H * max(dk, dv)))))
    layout = rng.choice(["bthd", "bhtd", "slices"])
    if layout == "slices":
        dv = dk
    packed = rng.randrange(2, 40) if B == 1 and T >= 64 and layout == "bthd" and rng.random() < 0.7 else 0
    gate = "head" if op == "prompt" and rng.random() < 0.25 else "token"
    return _attn(None, op, B, T, H, dk, dv, dtype, gate=gate, layout=layout, state0=rng.random() < 0.5, packed=packed,
                 resets=gate == "token" and rng.random() < 0.4)


# ---- inputs -------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _randn(gen, shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x if scale == 1.0 else x.mul_(scale)).to(dtype)


def _offsets(T, n, seed):
    """Offsets of n packed sequences over T steps; sequence 1 is empty, others of any length."""
    r = np.random.Generator(np.random.PCG64(int(seed) + 5))
    cuts = np.sort(r.integers(0, T + 1, n - 1))
    if n > 2:
        cuts[1] = cuts[0]
    return [0] + [int(c) for c in cuts] + [T]


def _decays(gen, shape, H, resets):
    """log sigmoid of a forget gate whose bias differs by head: memories of a few to some hundred steps."""
    bias = torch.linspace(1.0, 5.5, H, device="cuda")
    g = torch.nn.functional.logsigmoid(torch.randn(shape, generator=gen, device="cuda") + bias)
    if resets:  # a document starts: nothing before it is kept
        starts = torch.rand(shape[:-1], generator=gen, device="cuda") < 1.0 / 200.0
        g = g.masked_fill(starts[..., None], -math.inf)
    return g


def prepare(case, seed):
    c, gen = case, _gen(seed)
    dt = _DT[c["dtype"]]
    s = {"case": c}
    if c["op"].startswith("norm"):
        n, d = c["rows"], c["width"]
        s["x"] = (_randn(gen, (n, d)) * 1.5 + 0.25).to(dt)
        s["w"] = 1.0 + 0.1 * _randn(gen, (d,))
        s["b"] = 0.1 * _randn(gen, (d,))
        if c["op"] == "norm_backward":
            s["g"] = _randn(gen, (n, d), dt)
            x = s["x"].float()
            s["mean"] = x.mean(-1)
            s["rstd"] = (x.var(-1, unbiased=False) + _EPS).rsqrt()
        return s
    B, H, dk, dv = c["B"], c["H"], c["dk"], c["dv"]
    s["scale"] = dk ** -0.5
    if c["op"] == "step":
        s["q"], s["k"] = _randn(gen, (B, H, dk), dt), _randn(gen, (B, H, dk), dt)
        s["v"] = _randn(gen, (B, H, dv), dt)
        s["g"] = _decays(gen, (B, H), H, False)
        s["state"] = _randn(gen, (c["slots"], H, dk, dv))
        s["slots"] = torch.randperm(c["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        return s
    T = c["T"]
    if c["layout"] == "slices":  # one projection of (B, T, 4, H * d): q, k, v and a gate that is not read here
        P = _randn(gen, (B, T, 4, H * dk), dt)
        s["q"], s["k"], s["v"] = (P[:, :, i].view(B, T, H, dk) for i in range(3))
    elif c["layout"] == "bhtd":
        s["q"], s["k"], s["v"] = (_randn(gen, (B, H, T, d), dt).transpose(1, 2) for d in (dk, dk, dv))
    else:
        s["q"], s["k"], s["v"] = (_randn(gen, (B, T, H, d), dt) for d in (dk, dk, dv))
    if c["gate"] == "head":
        s["g"] = torch.nn.functional.logsigmoid(torch.linspace(1.0, 5.5, H, device="cuda"))
    else:
        s["g"] = _decays(gen, (B, T, H), H, c["resets"])
    n = c["packed"] or B
    s["cu"] = None
    if c["packed"]:
        at = _offsets(T, c["packed"], seed)
        s["cu"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        s["longest"] = max(b - a for a, b in zip(at, at[1:]))
    s["state0"] = _randn(gen, (n, H, dk, dv)) if c["state0"] else None
    if c["op"] == "train":
        s["do"] = _randn(gen, (B, T, H, dv), dt)
    return s


# ---- the plain forms ----------------------------------------------------------------------------
def _plain_norm(s):
    c = s["case"]
    x, w, b = s["x"].float(), s["w"], s["b"]
    if c["op"] == "norm_forward":
        mean = x.mean(-1)
        x = x - mean[:, None]
        rstd = (x.square().mean(-1) + _EPS).rsqrt()
        return (x * rstd[:, None] * w + b).to(_DT[c["out"]]), mean, rstd
    g = s["g"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gw = g * w
    dx = s["rstd"][:, None] * (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True))
    return dx.to(s["x"].dtype), (g * xh).sum(0), g.sum(0)


def _plain_step(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    idx = s["slots"].long()
    S = s["state"][idx] * torch.exp(s["g"])[..., None, None] + k[..., :, None] * v[..., None, :]
    s["state"][idx] = S
    o = (S * q[..., :, None]).sum(-2) * s["scale"]
    return o.to(s["q"].dtype), s["state"]


def _sums_between(g):
    """(..., n) -> (..., n, n): entry (i, j) is the sum of g over j+1 .. i, -inf where j > i."""
    n = g.shape[-1]
    i = torch.arange(n, device=g.device)
    x = g[..., :, None].expand(*g.shape, n).masked_fill(i[:, None] <= i[None, :], 0.0)
    return x.cumsum(-2).masked_fill(i[:, None] < i[None, :], -math.inf)


def _plain_attention(q, k, v, g, s0, C=64):
    """(B, H, T, d) float32 operands, g (B, H, T), s0 (B, H, dk, dv) or None -> (o, final state)."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    N = (T + C - 1) // C
    pad = N * C - T
    if pad:
        q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)) for x in (q, k, v))
        g = torch.nn.functional.pad(g, (0, pad))
    q, k, v = (x.reshape(B, H, N, C, -1) for x in (q, k, v))
    g = g.reshape(B, H, N, C)
    D = torch.exp(_sums_between(g))
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * D, v)
    kv = torch.matmul((k * D[..., -1, :, None]).transpose(-1, -2), v)  # what each chunk adds to the state
    first = torch.zeros(B, H, 1, dk, dv, device=q.device) if s0 is None else s0[:, :, None]
    E = torch.cat([first, kv], 2).reshape(B, H, N + 1, dk * dv)
    A = torch.cat([torch.zeros(B, H, 1, device=q.device), g.sum(-1)], 2)
    X = torch.matmul(torch.exp(_sums_between(A)), E).reshape(B, H, N + 1, dk, dv)
    o = o + torch.matmul(q, X[:, :, :-1]) * torch.exp(g.cumsum(-1))[..., None]
    return o.reshape(B, H, N * C, dv)[:, :, :T], X[:, :, -1]


def _apart(s):
    """Packed sequences as a padded batch: (index (S, L), inside (S, L)), or None."""
    cu = s["cu"]
    if cu is None:
        return None
    cu = cu.long()
    at = torch.arange(s["longest"], device=cu.device)
    inside = at[None] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(inside, cu[:-1, None] + at[None], s["case"]["T"]), inside


def _spread(x, apart):
    """(B, T, H, ...) operand to float32 (S, H, L, ...)."""
    x = x.float()
    if apart is not None:
        index, inside = apart
        x = x[0][index.clamp(max=x.shape[1] - 1)]
        x = torch.where(inside.reshape(inside.shape + (1,) * (x.dim() - 2)), x, 0.0)
    return x.transpose(1, 2)


def _join(x, apart, like, T):
    """(S, H, L, ...) back to (B, T, H, ...) of a type."""
    x = x.transpose(1, 2)
    if apart is not None:
        out = torch.zeros((T + 1,) + tuple(x.shape[2:]), device=x.device)
        out[apart[0]] = x  # steps outside a sequence land in the row past the last
        x = out[None, :T]
    return x.to(like).contiguous()


def _gates(s, apart):
    c = s["case"]
    g = s["g"].expand(c["B"], c["T"], c["H"]) if s["g"].dim() == 1 else s["g"]
    return _spread(g, apart)


def _plain_prompt(s):
    apart, dt, T = _apart(s), s["q"].dtype, s["case"]["T"]
    q, k, v = (_spread(s[n], apart) for n in "qkv")
    o, S = _plain_attention(q, k, v, _gates(s, apart), s["state0"])
    return _join(o * s["scale"], apart, dt, T), S


def _plain_train(s):
    apart, dt, T = _apart(s), s["q"].dtype, s["case"]["T"]
    q, k, v, do = (_spread(s[n], apart) for n in ("q", "k", "v", "do"))
    g, s0 = _gates(s, apart), s["state0"]
    qs = q * s["scale"]
    # backward in time a step's decay is that of the step after it; a padded tail adds nothing
    back = torch.nn.functional.pad(g.flip(-1)[..., :-1], (1, 0))
    qb, kb, vb, db = (x.flip(2) for x in (qs, k, v, do))
    dq = _plain_attention(do, v, k, g, None if s0 is None else s0.transpose(-1, -2))[0] * s["scale"]
    dk, L = (x for x in _plain_attention(vb, db, qb, back, None))
    dk = dk.flip(2)
    dv = _plain_attention(kb, qb, db, back, None)[0].flip(2)
    dg = ((q * dq).sum(-1) - (k * dk).sum(-1)).flip(-1).cumsum(-1).flip(-1)
    dg = torch.where(g == -math.inf, 0.0, dg)
    outs = [_join(dq, apart, dt, T), _join(dk, apart, dt, T), _join(dv, apart, dt, T),
            _join(dg, apart, torch.float32, T)]
    if s0 is not None:
        lead = torch.exp(g[..., 0])[..., None, None]
        outs.append(L.transpose(-1, -2) * lead)
    return outs


# ---- one pass -----------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if not own:
        if c["op"].startswith("norm"):
            return _plain_norm(s)
        return {"step": _plain_step, "prompt": _plain_prompt, "train": _plain_train}[c["op"]](s)
    global _lib
    if _lib is None:
        import recurrent_nets_amd as _lib
    if c["op"] == "norm_forward":
        return _lib.layer_norm_forward(s["x"], s["w"], s["b"], _EPS, out_dtype=_DT[c["out"]], want_stats=True)
    if c["op"] == "norm_backward":
        return _lib.layer_norm_backward(s["x"], s["g"], s["mean"], s["rstd"], s["w"])
    if c["op"] == "step":
        o = _lib.linear_attention_step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"], scale=s["scale"])
        return o, s["state"]
    if c["op"] == "prompt":
        return _lib.linear_attention_forward(s["q"], s["k"], s["v"], s["g"], s["state0"], scale=s["scale"],
                                             want_final_state=True, cu_seqlens=s["cu"])
    dq, dk, dv, dg, ds = _lib.linear_attention_backward(s["q"], s["k"], s["v"], s["g"], s["do"], s["state0"],
                                                        scale=s["scale"], want_dstate0=s["state0"] is not None,
                                                        cu_seqlens=s["cu"])
    return [dq, dk, dv, dg] + ([] if ds is None else [ds])


def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("norm"):
        n, d = c["rows"], c["width"]
        if c["op"] == "norm_forward":
            return {"bytes": n * d * (size + (2 if c["out"] == "bf16" else 4)) + 8 * n + 8 * d, "flops": 7 * n * d}
        return {"bytes": 3 * n * d * size + 8 * n + 12 * d, "flops": 14 * n * d}
    B, H, dk, dv = c["B"], c["H"], c["dk"], c["dv"]
    if c["op"] == "step":
        return {"bytes": B * H * (8 * dk * dv + size * 2 * (dk + dv) + 4) + 4 * B, "flops": 5 * B * H * dk * dv}
    tok = B * c["T"] * H
    n = (c["packed"] or B) * H
    gates = 4 * (H if c["gate"] == "head" else tok)
    if c["op"] == "prompt":
        return {"bytes": tok * size * 2 * (dk + dv) + gates + 4 * n * dk * dv * (2 if c["state0"] else 1),
                "flops": 4 * tok * dk * dv}
    return {"bytes": tok * size * (4 * dk + 3 * dv) + 2 * gates + (8 * n * dk * dv if c["state0"] else 0),
            "flops": 10 * tok * dk * dv}


# ---- from the definition, in 64 bits --------------------------------------------------------------
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"].startswith("norm"):
        x, w, b = (s[n].double() for n in ("x", "w", "b"))
        if c["op"] == "norm_forward":
            var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
            rstd = 1.0 / torch.sqrt(var + _EPS)
            return (x - mean) * rstd * w + b, mean[:, 0], rstd[:, 0]
        d, g = x.shape[1], s["g"].double()
        r = s["rstd"].double()[:, None]
        xh = (x - s["mean"].double()[:, None]) * r
        gw = g * w
        dx = (r / d) * (d * gw - gw.sum(1, keepdim=True) - xh * (gw * xh).sum(1, keepdim=True))
        return dx, torch.einsum("nd,nd->d", g, xh), g.sum(0)
    q, k, v = (s[n].double() for n in "qkv")
    if c["op"] == "step":
        o = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
        state = s["state"].double()
        for i, slot in enumerate(s["slots"].tolist()):
            S = state[slot] * s["g"][i].double().exp()[:, None, None] + torch.einsum("hk,hv->hkv", k[i], v[i])
            state[slot] = S
            o[i] = torch.einsum("hkv,hk->hv", S, q[i]) * s["scale"]
        return o, state
    T, H = c["T"], c["H"]
    g = s["g"].double().expand(c["B"], T, H)
    if c["packed"]:
        at = _offsets(T, c["packed"], seed)
        spans = [(0, a, b) for a, b in zip(at, at[1:])]
    else:
        spans = [(slice(None), 0, T)]
    total = sum(b - a for _, a, b in spans)
    if total * (3 if c["op"] == "train" else 1) * max(1e-4, c["B"] * H * c["dk"] * c["dv"] * 8 * 5 / 3e12) > 20:
        return None
    decay = g.exp()
    o, dq, dk_, dg = torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(g)
    dv_, ends, dstart = torch.zeros_like(v), [], []
    do = s["do"].double() if c["op"] == "train" else None
    for n, (rows, a, b) in enumerate(spans):
        pick = slice(n, n + 1) if c["packed"] else slice(None)
        row = slice(0, 1) if c["packed"] else rows
        m = 1 if c["packed"] else c["B"]
        S = torch.zeros(m, H, c["dk"], c["dv"], dtype=torch.float64, device="cuda")
        if s["state0"] is not None:
            S += s["state0"][pick].double()
        for t in range(a, b):
            S.mul_(decay[row, t][..., None, None]).add_(k[row, t][..., :, None] * v[row, t][..., None, :])
            if do is None:
                o[row, t] = torch.matmul(q[row, t][..., None, :], S)[..., 0, :] * s["scale"]
            else:
                dq[row, t] = torch.matmul(S, do[row, t][..., :, None])[..., 0] * s["scale"]
        ends.append(S)
        if do is None:
            continue
        L = torch.zeros_like(S)
        run_sum = torch.zeros(m, H, dtype=torch.float64, device="cuda")
        for t in range(b - 1, a - 1, -1):
            L.add_(q[row, t][..., :, None] * do[row, t][..., None, :] * s["scale"])
            dk_[row, t] = torch.matmul(L, v[row, t][..., :, None])[..., 0]
            dv_[row, t] = torch.matmul(k[row, t][..., None, :], L)[..., 0, :]
            run_sum = run_sum + (q[row, t] * dq[row, t]).sum(-1) - (k[row, t] * dk_[row, t]).sum(-1)
            dg[row, t] = torch.where(decay[row, t] == 0, 0.0, run_sum)
            L.mul_(decay[row, t][..., None, None])
        dstart.append(L)
    if do is None:
        return o, torch.cat(ends)
    outs = [dq, dk_, dv_, dg]
    return outs + ([torch.cat(dstart)] if s["state0"] is not None else [])
