"""The token operators beside the Nystrom attention, as they are measured: decay attention (prompt,
backward, single-token step), rotary positions, and group norm with an activation.

Shapes are [B, heads, N, d] for attention tensors (memory order "bhnd", or "bnhd" as a projection
leaves them), [B, N, C] for the norm. Cases name an operator ("op") and its sizes.
"""
from __future__ import annotations

import math

import torch

own = False

CHUNK = 64   # tokens per block of the plain prompt form


def listed():
    return [
        # one short prompt of one user: launch latency
        dict(name="prompt short", op="decay_fwd", dtype="bf16", B=1, heads=8, N=113, dk=64, dv=64,
             order="bnhd", state=False, ragged=False),
        # one long sequence continued from a state (256 x 256 tokens, the long workload's size): few units
        dict(name="prompt long", op="decay_fwd", dtype="bf16", B=1, heads=8, N=65536, dk=64, dv=64,
             order="bhnd", state=True, ragged=False),
        # a padded batch of prompts with wide heads, as a projection lays them out
        dict(name="prompt batch", op="decay_fwd", dtype="bf16", B=8, heads=16, N=4096, dk=128, dv=128,
             order="bnhd", state=True, ragged=True),
        # full-precision training at the stage-2 token count, narrow keys
        dict(name="prompt fp32", op="decay_fwd", dtype="f32", B=32, heads=2, N=784, dk=32, dv=64,
             order="bhnd", state=False, ragged=False),
        # training step of a batch of sequences
        dict(name="backward batch", op="decay_bwd", dtype="bf16", B=8, heads=16, N=2048, dk=128, dv=128,
             order="bnhd", state=False, ragged=False),
        # training step on high-resolution grids (112 x 112 tokens) minus a ragged tail, through a state
        dict(name="backward ragged", op="decay_bwd", dtype="bf16", B=4, heads=2, N=12544, dk=64, dv=64,
             order="bhnd", state=True, ragged=True),
        # one generated token of one user: launch latency
        dict(name="step single", op="decay_step", dtype="bf16", B=1, heads=8, dk=64, dv=64),
        # one generated token of many users, states in a pool
        dict(name="step batch", op="decay_step", dtype="bf16", B=192, heads=16, dk=128, dv=128),
        # positions on q and k of a batch of prompts, part of the head, stretched context
        dict(name="rotary prompt", op="rotary", dtype="bf16", B=4, heads=16, heads2=16, N=4096, d=128, rot=96,
             layout="half", scaling=4.0, inverse=False, order="bnhd"),
        # gradients of rotated full-precision q and k at single far positions
        dict(name="rotary far", op="rotary", dtype="f32", B=64, heads=8, heads2=8, N=1, d=64, rot=64,
             layout="interleaved", scaling=1.0, inverse=True, order="bhnd"),
        # norm of every head's output of every token (one sample per token)
        dict(name="norm heads", op="norm_fwd", dtype="bf16", B=8192, N=1, C=1024, groups=16, act="silu"),
        # training step of the norm on stage-1 token maps (56 x 56), forward saved
        dict(name="norm backward", op="norm_bwd", dtype="bf16", B=32, N=3136, C=256, groups=32, act="silu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decay_fwd", "decay_fwd", "decay_bwd", "decay_bwd", "decay_step", "rotary", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("decay_fwd", "decay_bwd"):
        dk, dv = (8 * rng.randint(2, 16) for _ in range(2))
        # at most the largest listed case's tokens (fp32 on a quarter of them)
        units = _log_int(rng, 1, 128)
        heads = rng.choice([h for h in (1, 2, 4, 6, 8, 16) if h <= units])
        B = max(1, units // heads)
        most = (8 * 16 * 4096 if op == "decay_fwd" else 8 * 16 * 2048) // (1 if dtype == "bf16" else 4)
        N = _log_int(rng, 1, max(1, min(65536 if op == "decay_fwd" else 16384, most // (B * heads))))
        return dict(op=op, dtype=dtype, B=B, heads=heads, N=N, dk=dk, dv=dv, order=rng.choice(["bhnd", "bnhd"]),
                    state=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "decay_step":
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 192), heads=rng.randint(1, 16),
                    dk=8 * rng.randint(2, 16), dv=8 * rng.randint(2, 16))
    if op == "rotary":
        d = 8 * rng.randint(4, 16)
        heads, heads2 = rng.randint(1, 16), rng.choice([0, 1, 2, 4, 8, 16])
        B = _log_int(rng, 1, 64)
        N = _log_int(rng, 1, max(1, 4 * 4096 * 32 // (B * (heads + heads2))))
        return dict(op=op, dtype=dtype, B=B, heads=heads, heads2=heads2, N=min(N, 65536), d=d,
                    rot=2 * rng.randint(4, d // 2), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice([1.0, 4.0, 16.0]), inverse=rng.random() < 0.5,
                    order=rng.choice(["bhnd", "bnhd"]))
    groups = rng.choice([1, 2, 4, 8, 16, 32])
    C = groups * rng.choice([4, 8, 10, 16, 24, 64, 72])
    most = 32 * 3136 * 256 // (1 if dtype == "bf16" else 2)
    N = _log_int(rng, 1, min(16384, max(1, most // C)))
    B = _log_int(rng, 1, max(1, min(8192, most // (C * N))))
    return dict(op=op, dtype=dtype, B=B, N=N, C=C, groups=groups, act=rng.choice(["none", "silu", "gelu"]))


# ---- inputs ------------------------------------------------------------------------------------

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _tokens(g, case, heads, d, fill=None):
    """A [B, heads, N, d] tensor in the case's memory order."""
    B, N = case["B"], case["N"]
    shape = (B, heads, N, d) if case["order"] == "bhnd" else (B, N, heads, d)
    t = torch.zeros(shape, device="cuda", dtype=_type(case)) if fill == 0 else \
        torch.randn(shape, device="cuda", generator=g).to(_type(case))
    return t if case["order"] == "bhnd" else t.transpose(1, 2)


def _log_decay(heads):
    """Decays 1 - 2^-5 .. 1 - 2^-12 over the heads."""
    e = torch.linspace(-5.0, -12.0, heads, dtype=torch.float64) if heads > 1 else torch.tensor([-8.0], dtype=torch.float64)
    return torch.log1p(-torch.exp2(e)).float().cuda()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op in ("decay_fwd", "decay_bwd"):
        B, heads, N, dk, dv = (case[k] for k in ("B", "heads", "N", "dk", "dv"))
        s["q"], s["k"], s["v"] = _tokens(g, case, heads, dk), _tokens(g, case, heads, dk), _tokens(g, case, heads, dv)
        s["log_decay"], s["scale"] = _log_decay(heads), dk ** -0.5
        s["S0"] = torch.randn((B, heads, dk, dv), device="cuda", generator=g) if case["state"] else None
        s["lengths"] = None
        if case["ragged"]:
            at = torch.randint(max(1, N // 2), N + 1, (B,), device="cuda", generator=g)
            s["lengths"] = at.to(torch.int32)
        if op == "decay_fwd":
            s["O"] = _tokens(g, case, heads, dv, fill=0)
            s["S_out"] = torch.zeros((B, heads, dk, dv), device="cuda") if case["state"] else None
        else:
            s["dO"] = _tokens(g, case, heads, dv)
            s["dS_out"] = torch.randn((B, heads, dk, dv), device="cuda", generator=g) if case["state"] else None
            s["dQ"], s["dK"], s["dV"] = (_tokens(g, case, heads, d, fill=0) for d in (dk, dk, dv))
            s["dS0"] = torch.zeros((B, heads, dk, dv), device="cuda") if case["state"] else None
    elif op == "decay_step":
        B, heads, dk, dv = (case[k] for k in ("B", "heads", "dk", "dv"))
        s["q"], s["k"], s["v"] = (torch.randn((B, heads, d), device="cuda", generator=g).to(_type(case)) for d in (dk, dk, dv))
        s["log_decay"], s["scale"] = _log_decay(heads), dk ** -0.5
        s["S"] = torch.randn((B, heads, dk, dv), device="cuda", generator=g)
        s["slots"] = torch.randperm(B, device="cuda", generator=g).to(torch.int32)   # states in a pool's order
        s["O"] = torch.zeros((B, heads, dv), device="cuda", dtype=_type(case))
    elif op == "rotary":
        s["x"] = _tokens(g, case, case["heads"], case["d"])
        s["x2"] = _tokens(g, case, case["heads2"], case["d"]) if case["heads2"] else None
        s["y"] = _tokens(g, case, case["heads"], case["d"], fill=0)
        s["y2"] = _tokens(g, case, case["heads2"], case["d"], fill=0) if case["heads2"] else None
        first = torch.randint(0, 200000, (case["B"], 1), device="cuda", generator=g)   # far into a conversation
        s["positions"] = (first + torch.arange(case["N"], device="cuda")).to(torch.int32)
        i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
        s["freqs"] = 10000.0 ** (-2.0 * i / case["rot"]) / case["scaling"]
        s["mscale"] = 0.1 * math.log(case["scaling"]) + 1.0
    else:
        B, N, C = case["B"], case["N"], case["C"]
        s["x"] = (torch.randn((B, N, C), device="cuda", generator=g) + 0.5).to(_type(case))
        s["gamma"] = 1.0 + 0.2 * torch.randn((C,), device="cuda", generator=g)
        s["beta"] = 0.2 * torch.randn((C,), device="cuda", generator=g)
        s["eps"] = 1e-5
        if op == "norm_fwd":
            s["y"] = torch.zeros_like(s["x"])
        else:
            s["dy"] = torch.randn((B, N, C), device="cuda", generator=g).to(_type(case))
            s["dx"] = torch.zeros_like(s["x"])
            x = s["x"].view(B, N, case["groups"], -1).double()
            m = x.mean((1, 3))
            s["mean"] = m.float()
            s["rstd"] = (((x - m[:, None, :, None]) ** 2).mean((1, 3)) + s["eps"]).rsqrt().float()
    return s


# ---- plain forms -------------------------------------------------------------------------------

def _blocks(t, valid):
    """[B, heads, N, d] -> fp32 [B, heads, blocks, CHUNK, d], zeros behind each sequence's end."""
    t = torch.where(valid[:, None, :, None], t.float(), torch.zeros((), device=t.device))
    pad = -t.shape[2] % CHUNK
    t = torch.nn.functional.pad(t, (0, 0, 0, pad))
    return t.reshape(t.shape[0], t.shape[1], -1, CHUNK, t.shape[3])


def _valid(s):
    n = torch.arange(s["case"]["N"], device="cuda")
    if s["lengths"] is None:
        return torch.ones((s["case"]["B"], 1), device="cuda", dtype=torch.bool).expand(-1, n.numel())
    return n[None, :] < s["lengths"][:, None]


def _power(log_decay, n):
    """decay^n for whole n >= 0 (0 where n < 0), [heads, *n.shape]."""
    p = torch.exp(log_decay.reshape(-1, *([1] * n.dim())).double() * n.clamp(min=0)).float()
    return torch.where(n < 0, torch.zeros((), device=n.device), p)


def _carried(log_decay, local, first):
    """States before each block from the blocks' own sums [B, heads, blocks, dk, dv], already decayed
    to each block's end, and the state before the first."""
    n = torch.arange(local.shape[2], device="cuda")
    w = _power(log_decay * CHUNK, (n[:, None] - 1) - n[None, :])
    before = torch.matmul(w, local.flatten(3)).view(local.shape)
    return before if first is None else before + _power(log_decay * CHUNK, n)[None, :, :, None, None] * first[:, :, None]


def _attend(s, q, k, v, first):
    """The causal form in blocks: outputs of every position and the blocks' own sums."""
    i = torch.arange(CHUNK, device="cuda")
    ld = s["log_decay"]
    local = torch.matmul((k * _power(ld, CHUNK - 1 - i)[None, :, None, :, None]).transpose(-1, -2), v)
    before = _carried(ld, local, first)
    a = torch.matmul(q, k.transpose(-1, -2)) * _power(ld, i[:, None] - i[None, :])[None, :, None]
    return torch.matmul(a, v) + torch.matmul(q * _power(ld, i + 1)[None, :, None, :, None], before)


def _from_blocks(t, case, like):
    return t.reshape(t.shape[0], t.shape[1], -1, t.shape[4])[:, :, :case["N"]].to(like.dtype)


def _decay_fwd(s):
    case, valid, ld = s["case"], _valid(s), s["log_decay"]
    q, k, v = (_blocks(s[n], valid) for n in "qkv")
    o = _from_blocks(s["scale"] * _attend(s, q, k, v, s["S0"]), case, s["q"])
    o = torch.where(valid[:, None, :, None], o, torch.zeros((), device="cuda", dtype=o.dtype))
    if not case["state"]:
        return dict(o=o)
    length = valid.sum(1)
    left = length[:, None] - 1 - torch.arange(case["N"], device="cuda")[None, :]            # [B, N]
    w = _power(ld, left).permute(1, 0, 2)[..., None]                                          # [B, heads, N, 1]
    kv = torch.where(valid[:, None, :, None], s["k"].float() * w, torch.zeros((), device="cuda"))
    vv = torch.where(valid[:, None, :, None], s["v"].float(), torch.zeros((), device="cuda"))
    S = torch.matmul(kv.transpose(-1, -2), vv) + _power(ld, length).t()[..., None, None] * s["S0"]
    return dict(o=o, S=S)


def _decay_bwd(s):
    case, valid, ld = s["case"], _valid(s), s["log_decay"]
    zero = torch.zeros((), device="cuda")
    q, k, v, do = (_blocks(s[n], valid) for n in ("q", "k", "v", "dO"))
    # dq: the same causal form, queries do, keys v, values k, state transposed
    first = None if s["S0"] is None else s["S0"].transpose(-1, -2)
    dq = s["scale"] * _attend(s, do, v, k, first)
    # dk, dv: the same from the sequence's end; the end's gradient enters undecayed
    back = [t.flip((2, 3)) for t in (q, k, v, do)]
    dk = s["scale"] * _attend(s, back[2], back[3], back[0], None).flip((2, 3))
    dv = s["scale"] * _attend(s, back[1], back[0], back[3], None).flip((2, 3))
    dq, dk, dv = (_from_blocks(t, case, zero) for t in (dq, dk, dv))
    out = {}
    if s["dS_out"] is not None:
        length, n = valid.sum(1), torch.arange(case["N"], device="cuda")
        w = _power(ld, length[:, None] - 1 - n[None, :]).permute(1, 0, 2)[..., None]
        dk = dk + w * torch.matmul(s["v"].float(), s["dS_out"].transpose(-1, -2))
        dv = dv + w * torch.matmul(s["k"].float(), s["dS_out"])
        wq = _power(ld, n + 1)[None, :, :, None]
        qs = torch.where(valid[:, None, :, None], s["q"].float() * wq, zero)
        dos = torch.where(valid[:, None, :, None], s["dO"].float(), zero)
        out["dS0"] = s["scale"] * torch.matmul(qs.transpose(-1, -2), dos) + \
            _power(ld, length).t()[..., None, None] * s["dS_out"]
    return dict(out, **{name: torch.where(valid[:, None, :, None], t, zero).to(s["q"].dtype)
                        for name, t in (("dq", dq), ("dk", dk), ("dv", dv))})


def _decay_step(s):
    at = s["slots"].long()
    S = torch.exp(s["log_decay"])[:, None, None] * s["S"][at] + s["k"].float()[..., None] * s["v"].float()[..., None, :]
    s["S"][at] = S
    o = s["scale"] * torch.matmul(s["q"].float()[..., None, :], S).squeeze(-2)
    return dict(o=o.to(s["q"].dtype), S=s["S"])


def _rotate(s, x):
    case, rot = s["case"], s["case"]["rot"]
    angle = s["positions"].double()[:, None, :, None] * s["freqs"]
    c, n = (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()
    if case["inverse"]:
        n = -n
    t, rest = x[..., :rot].float(), x[..., rot:]
    if case["layout"] == "half":
        a, b = t[..., :rot // 2], t[..., rot // 2:]
        r = torch.cat((a * c - b * n, a * n + b * c), -1)
    else:
        a, b = t[..., 0::2], t[..., 1::2]
        r = torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)
    return torch.cat((r.to(x.dtype), rest), -1)


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _act_slope(z, act):
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    return torch.ones_like(z)


def _norm_fwd(s):
    case, shape = s["case"], s["x"].shape
    x = s["x"].float().view(case["B"], case["N"], case["groups"], -1)
    mean = x.mean((1, 3))
    xc = x - mean[:, None, :, None]
    rstd = ((xc * xc).mean((1, 3)) + s["eps"]).rsqrt()
    z = (xc * rstd[:, None, :, None]).view(shape) * s["gamma"] + s["beta"]
    return dict(y=_act(z, case["act"]).to(s["x"].dtype), mean=mean, rstd=rstd)


def _norm_bwd(s):
    case, shape = s["case"], s["x"].shape
    grouped = (case["B"], case["N"], case["groups"], -1)
    rstd = s["rstd"][:, None, :, None]
    xh = (s["x"].float().view(grouped) - s["mean"][:, None, :, None]) * rstd
    dz = s["dy"].float() * _act_slope(xh.view(shape) * s["gamma"] + s["beta"], case["act"])
    g = (dz * s["gamma"]).view(grouped)
    dx = rstd * (g - g.mean((1, 3), keepdim=True) - xh * (g * xh).mean((1, 3), keepdim=True))
    return dict(dx=dx.reshape(shape).to(s["x"].dtype), dgamma=(dz * xh.view(shape)).sum((0, 1)), dbeta=dz.sum((0, 1)))


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        return _own(s)
    if op == "decay_fwd":
        return _decay_fwd(s)
    if op == "decay_bwd":
        return _decay_bwd(s)
    if op == "decay_step":
        return _decay_step(s)
    if op == "rotary":
        y = dict(y=_rotate(s, s["x"]))
        return y if s["x2"] is None else dict(y, y2=_rotate(s, s["x2"]))
    return _norm_fwd(s) if op == "norm_fwd" else _norm_bwd(s)


def _own(s):
    from laplacian_nystr_attention_avg_b200 import decay

    case = s["case"]
    op = case["op"]
    if op == "decay_fwd":
        o, S = decay.decay_forward(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], S0=s["S0"],
                                   lengths=s["lengths"], O=s["O"], S_out=s["S_out"])
        return dict(o=o) if S is None else dict(o=o, S=S)
    if op == "decay_bwd":
        dq, dk, dv, dS0 = decay.decay_backward(s["q"], s["k"], s["v"], s["log_decay"], s["dO"], scale=s["scale"],
                                               S0=s["S0"], lengths=s["lengths"], dS_out=s["dS_out"], dQ=s["dQ"],
                                               dK=s["dK"], dV=s["dV"], dS0=s["dS0"])
        return dict(dq=dq, dk=dk, dv=dv) if dS0 is None else dict(dq=dq, dk=dk, dv=dv, dS0=dS0)
    if op == "decay_step":
        o = decay.decay_step(s["q"], s["k"], s["v"], s["log_decay"], s["S"], scale=s["scale"], slots=s["slots"], O=s["O"])
        return dict(o=o, S=s["S"])
    if op == "rotary":
        y, y2 = decay.rotary(s["x"], s["positions"], s["freqs"], x2=s["x2"], layout=case["layout"],
                             mscale=s["mscale"], inverse=case["inverse"], out=s["y"], out2=s["y2"])
        return dict(y=y) if y2 is None else dict(y=y, y2=y2)
    if op == "norm_fwd":
        y, mean, rstd = decay.group_norm(s["x"], case["groups"], s["gamma"], s["beta"], eps=s["eps"], act=case["act"], out=s["y"])
        return dict(y=y, mean=mean, rstd=rstd)
    dx, dgamma, dbeta = decay.group_norm_backward(s["x"], s["dy"], s["mean"], s["rstd"], case["groups"], s["gamma"],
                                                  s["beta"], act=case["act"], dx=s["dx"])
    return dict(dx=dx, dgamma=dgamma, dbeta=dbeta)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    e, op = 2 if case["dtype"] == "bf16" else 4, case["op"]
    if op in ("decay_fwd", "decay_bwd"):
        units, dk, dv = case["B"] * case["heads"], case["dk"], case["dv"]
        tokens = units * case["N"] * (0.75 if case["ragged"] else 1.0)
        states = 4 * units * dk * dv if case["state"] else 0
        if op == "decay_fwd":
            return {"bytes": e * tokens * (2 * dk + 2 * dv) + 2 * states, "flops": 4 * tokens * dk * dv}
        return {"bytes": e * tokens * (4 * dk + 3 * dv) + 3 * states, "flops": 10 * tokens * dk * dv}
    if op == "decay_step":
        units, dk, dv = case["B"] * case["heads"], case["dk"], case["dv"]
        return {"bytes": units * (8 * dk * dv + e * (2 * dk + 2 * dv)), "flops": 5 * units * dk * dv}
    if op == "rotary":
        n = case["B"] * (case["heads"] + case["heads2"]) * case["N"]
        return {"bytes": 2 * e * n * case["d"] + 4 * case["B"] * case["N"], "flops": 3 * n * case["rot"]}
    n = case["B"] * case["N"] * case["C"]
    return {"bytes": (2 if op == "norm_fwd" else 3) * e * n, "flops": (8 if op == "norm_fwd" else 20) * n}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def recurrence(backward):
        """The recurrence token by token."""
        B, H, N, dk, dv = (case[k] for k in ("B", "heads", "N", "dk", "dv"))
        lam = s["log_decay"].double().exp()[None, :, None, None]
        at = torch.full((B,), N, device="cuda") if s["lengths"] is None else s["lengths"].long()
        q, k, v = (s[n].permute(2, 0, 1, 3).contiguous() for n in "qkv")
        on = (torch.arange(N, device="cuda")[:, None] < at[None, :]).double()[:, :, None, None]
        S = torch.zeros((B, H, dk, dv), device="cuda", dtype=torch.float64) if s["S0"] is None else s["S0"].double()
        do = s["dO"].permute(2, 0, 1, 3).contiguous() if backward else None
        rows = torch.zeros((N, B, H, dk if backward else dv), device="cuda", dtype=torch.float64)
        for t in range(N):
            kt, vt = k[t].double().view(B * H, dk, 1), v[t].double().view(B * H, 1, dv)
            new = torch.baddbmm((S * lam).view(B * H, dk, dv), kt, vt).view_as(S)
            S = torch.lerp(S, new, on[t][..., None]) if s["lengths"] is not None else new
            r = torch.matmul(S, do[t].double()[..., None])[..., 0] if backward else torch.matmul(q[t].double()[..., None, :], S)[..., 0, :]
            rows[t] = s["scale"] * r * on[t]
        rows = rows.permute(1, 2, 0, 3)
        if not backward:
            return dict(o=rows, S=S) if case["state"] else dict(o=rows)
        G = torch.zeros_like(S) if s["dS_out"] is None else s["dS_out"].double()   # what reaches S_t from later tokens
        dks, dvs = (torch.zeros((N, B, H, d), device="cuda", dtype=torch.float64) for d in (dk, dv))
        for t in range(N - 1, -1, -1):
            qt, dot = s["scale"] * q[t].double().view(B * H, dk, 1), do[t].double().view(B * H, 1, dv)
            G1 = torch.baddbmm(G.view(B * H, dk, dv), qt, dot).view_as(S)
            dks[t] = torch.matmul(G1, v[t].double()[..., None])[..., 0] * on[t]
            dvs[t] = torch.matmul(k[t].double()[..., None, :], G1)[..., 0, :] * on[t]
            G = torch.lerp(G, G1 * lam, on[t][..., None]) if s["lengths"] is not None else G1 * lam
        out = dict(dq=rows, dk=dks.permute(1, 2, 0, 3), dv=dvs.permute(1, 2, 0, 3))
        return dict(out, dS0=G) if case["state"] else out

    if op in ("decay_fwd", "decay_bwd"):
        # about 0.15 ms a token for small states, and the state's own traffic for many
        each = 1.5e-4 + case["B"] * case["heads"] * case["dk"] * case["dv"] * 8 * 8 / 4e12
        return recurrence(op == "decay_bwd") if each * case["N"] * (2 if op == "decay_bwd" else 1) < 15 else None
    if op == "decay_step":
        S, at = s["S"].double(), s["slots"].long()
        lam = s["log_decay"].double().exp()
        new = torch.einsum("h,bhij->bhij", lam, S[at]) + torch.einsum("bhi,bhj->bhij", s["k"].double(), s["v"].double())
        S[at] = new
        return dict(o=s["scale"] * torch.einsum("bhi,bhij->bhj", s["q"].double(), new), S=S)
    if op == "rotary":
        w = torch.polar(torch.full((), s["mscale"], device="cuda", dtype=torch.float64),
                        s["positions"].double()[..., None] * s["freqs"] * (-1 if case["inverse"] else 1))[:, None]
        out = {}
        for name, x in (("y", s["x"]), ("y2", s["x2"])):
            if x is not None:
                y, h = x.double().clone(), case["rot"] // 2
                first, second = (slice(0, h), slice(h, 2 * h)) if case["layout"] == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
                z = torch.complex(y[..., first], y[..., second]) * w
                y[..., first], y[..., second] = z.real, z.imag
                out[name] = y
        return out
    x = s["x"].double().unflatten(2, (case["groups"], -1))
    var, mean = torch.var_mean(x, dim=(1, 3), correction=0, keepdim=True)
    rstd = 1 / torch.sqrt(var + s["eps"])
    xh = ((x - mean) * rstd).flatten(2).requires_grad_()
    z = xh * s["gamma"].double() + s["beta"].double()
    act = dict(none=lambda t: t, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu)[case["act"]]
    y = act(z)
    if op == "norm_fwd":
        return dict(y=y.detach(), mean=mean[:, 0, :, 0], rstd=rstd[:, 0, :, 0])
    dy = s["dy"].double()
    dxh, = torch.autograd.grad(y, xh, dy)
    dz = dxh / s["gamma"].double()
    d, h = dxh.unflatten(2, (case["groups"], -1)), xh.detach().unflatten(2, (case["groups"], -1))
    dx = rstd * (d - d.mean((1, 3), keepdim=True) - h * (d * h).mean((1, 3), keepdim=True))
    return dict(dx=dx.flatten(2), dgamma=(dz * xh.detach()).sum((0, 1)), dbeta=dz.sum((0, 1)))
