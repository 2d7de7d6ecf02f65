"""Cases of the operators around the GKA layer: the block's norms and gates before
the layer (``block_in``), the gated linear recurrence (``linear``, its backward
``linear_grad`` and its single-token step ``linear_step``) and the block's gated
norm after the layer (``block_out``), with the backward of both block parts.

Definitions (per batch b, head h, token t):
  block_in   qh = q rsqrt(|q|^2 + eps), kh likewise, v as it is, from [B, T, heads, D]
             rows to [B, H, T, D], key/value heads repeated over their group;
             beta = sigmoid(beta_logit + beta_bias_h), gate likewise; tokens at or
             past lengths[b] become zero rows with beta = 1, gate = 0
  linear     M_t = beta_t M_{t-1} + g_t v_t k_t^T,  o_t = scale M_t q_t
  block_out  u = o + skip_h v,  y = u rsqrt(mean u^2 + eps) w silu(z), back to [B, T, H, D]
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
# Plain forms work on chunks of this many tokens.
_CHUNK = 128
# Smallest decay the plain backward distinguishes from zero: contributions through a smaller
# one are below 2^-60 of what was written, and dbeta stays a quotient of normal numbers.
_BETA_MIN = 2.0 ** -60


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _rows(op, dtype, B, T, H, Hk, D, gate, lengths):
    return {"op": op, "dtype": dtype, "B": B, "T": T, "H": H, "Hk": Hk, "D": D, "gate": gate,
            "lengths": lengths}


def _lin(op, dtype, B, H, T, D, gate, state, resets):
    return {"op": op, "dtype": dtype, "B": B, "H": H, "T": T, "D": D, "gate": gate, "state": state,
            "resets": resets}


def _out(op, dtype, B, T, H, D, z, skip):
    return {"op": op, "dtype": dtype, "B": B, "T": T, "H": H, "D": D, "z": z, "skip": skip}


def listed():
    return [
        # the default training shape's projections, on their way into the layer
        dict(_rows("block_in", "bf16", 8, 2048, 8, 8, 128, True, False), name="in_bf16_b8t2048h8d128"),
        # gradient of a padded batch with shared key/value heads and an odd length
        dict(_rows("block_in_grad", "bf16", 6, 1021, 16, 4, 64, True, True),
             name="in_grad_bf16_b6t1021h16k4d64"),
        # one token of a small batch: what a served request needs (launch latency)
        dict(_lin("linear_step", "bf16", 1, 8, 1, 128, False, True, False), name="step_bf16_b1h8d128"),
        # the decode workload's batch: the state's traffic is all there is
        dict(_lin("linear_step", "bf16", 256, 32, 1, 128, True, True, False),
             name="step_bf16_b256h32d128"),
        # the small fp32 workload
        dict(_lin("linear", "fp32", 1, 2, 256, 32, False, False, False), name="linear_fp32_b1h2t256d32"),
        # the default training shape
        dict(_lin("linear", "bf16", 8, 8, 2048, 128, False, False, False),
             name="linear_bf16_b8h8t2048d128"),
        # a prompt that goes on from a cached state, packed documents (resets), one token short
        # of whole chunks
        dict(_lin("linear", "bf16", 4, 16, 8191, 128, True, True, True),
             name="linear_bf16_b4h16t8191d128"),
        # a long context with few heads
        dict(_lin("linear", "bf16", 1, 8, 131072, 128, False, False, False),
             name="linear_bf16_b1h8t131072d128"),
        # training step of the default shape
        dict(_lin("linear_grad", "bf16", 8, 8, 2048, 128, False, False, False),
             name="linear_grad_bf16_b8h8t2048d128"),
        # fp32 gradient, odd length, write gate, state and resets
        dict(_lin("linear_grad", "fp32", 2, 4, 517, 64, True, True, True),
             name="linear_grad_fp32_b2h4t517d64"),
        # fp32 output norm without gate or residual
        dict(_out("block_out", "fp32", 2, 509, 4, 32, False, False), name="out_fp32_b2t509h4d32"),
        # gradient of the output norm at the default training shape
        dict(_out("block_out_grad", "bf16", 8, 2048, 8, 128, True, True),
             name="out_grad_bf16_b8t2048h8d128"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["block_in", "block_in_grad", "linear", "linear", "linear", "linear_grad",
                     "linear_grad", "linear_step", "block_out", "block_out_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    D = rng.choice([32, 64, 128, 128])
    if op == "linear_step":
        return _lin(op, dtype, _log_int(rng, 1, 256), rng.randint(1, 32), 1, D, rng.random() < 0.5, True,
                    False)
    if op in ("linear", "linear_grad"):
        # head tokens: the long context's for the forward, the training shape's for the gradient
        most = 1 << 20 if op == "linear" else 1 << 17
        if dtype == "fp32":
            most >>= 2
        T = _log_int(rng, 1, 131072 if op == "linear" else 16384)
        T = min(T, most)
        H = _log_int(rng, 1, min(32, max(1, most // T)))
        B = _log_int(rng, 1, min(16, max(1, most // (T * H))))
        return _lin(op, dtype, B, H, T, D, rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5)
    T = _log_int(rng, 1, 8192)
    B = _log_int(rng, 1, 16)
    if op.startswith("block_in"):
        Hk = rng.choice([1, 2, 4, 8])
        H = Hk * rng.choice([1, 1, 2, 4])
        T = max(1, min(T, (1 << 18) // (B * H)))
        return _rows(op, dtype, B, T, H, Hk, D, rng.random() < 0.7, rng.random() < 0.5)
    H = rng.randint(1, 32)
    T = max(1, min(T, (1 << 18) // (B * H)))
    return _out(op, dtype, B, T, H, D, rng.random() < 0.7, rng.random() < 0.5)


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[case["dtype"]]
    B, T, H, D = case["B"], case["T"], case["H"], case["D"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": case, "dt": dt}
    op = case["op"]
    if op.startswith("block_in"):
        Hk = case["Hk"]
        # one projection's output: q, k, v side by side in every token's row
        qkv = randn(B, T, (H + 2 * Hk) * D).to(dt)
        ba = randn(B, T, 2 * H).to(dt)
        s["q"] = qkv[..., :H * D].unflatten(-1, (H, D))
        s["k"] = qkv[..., H * D:(H + Hk) * D].unflatten(-1, (Hk, D))
        s["v"] = qkv[..., (H + Hk) * D:].unflatten(-1, (Hk, D))
        s["beta_logit"] = ba[..., :H]
        s["gate_logit"] = ba[..., H:] if case["gate"] else None
        s["beta_bias"] = 3.0 + 0.5 * randn(H)
        s["gate_bias"] = 0.5 * randn(H) if case["gate"] else None
        s["lengths"] = None
        if case["lengths"]:
            # the first sequence is whole, another may be empty
            n = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
            n[0] = T
            s["lengths"] = n
        if op == "block_in_grad":
            for n in ("dq", "dk", "dv"):
                s[n] = randn(B, H, T, D).to(dt)
            s["dbeta"] = randn(B, H, T)
            s["dgate"] = randn(B, H, T) if case["gate"] else None
    elif op.startswith("linear"):
        step = op == "linear_step"
        shape = (B, H, D) if step else (B, H, T, D)
        for n in ("q", "k"):
            x = randn(*shape)
            s[n] = (x * torch.rsqrt((x * x).sum(-1, keepdim=True))).to(dt)
        s["v"] = randn(*shape).to(dt)
        s["beta"] = torch.sigmoid(3.0 + randn(*shape[:-1]))
        if case["resets"]:
            # a new document starts at about one token in 300
            u = torch.rand(*shape[:-1], generator=g, device=dev)
            s["beta"] = s["beta"].masked_fill(u < 1.0 / 300.0, 0.0)
        s["gate"] = torch.sigmoid(1.5 * randn(*shape[:-1])) if case["gate"] else None
        s["scale"] = D ** -0.5
        s["state"] = randn(B, H, D, D) if case["state"] else None
        if op == "linear_grad":
            s["dout"] = randn(*shape).to(dt)
            s["dfinal"] = randn(B, H, D, D) if case["state"] else None
    else:
        s["o"] = randn(B, H, T, D).to(dt)
        s["w"] = 1.0 + 0.1 * randn(D)
        s["z"] = randn(B, T, H, D).to(dt) if case["z"] else None
        s["v"] = randn(B, H, T, D).to(dt) if case["skip"] else None
        s["skip"] = 1.0 + 0.1 * randn(H) if case["skip"] else None
        if op == "block_out_grad":
            s["dy"] = randn(B, T, H, D).to(dt)
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _valid(s):
    """[B, 1, T] truth values of the tokens inside their sequence, or None."""
    if s["lengths"] is None:
        return None
    t = torch.arange(s["case"]["T"], device=s["lengths"].device)
    return (t[None, :] < s["lengths"][:, None])[:, None, :]


def _block_in_plain(s):
    dt, rep = s["dt"], s["case"]["H"] // s["case"]["Hk"]
    ok = _valid(s)

    def rows(x, unit, n):
        x = x.float()
        if unit:
            x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)
        x = x.permute(0, 2, 1, 3).repeat_interleave(n, 1)
        if ok is not None:
            x = torch.where(ok[..., None], x, 0.0)
        return x.to(dt).contiguous()

    def gates(logit, bias, pad):
        x = torch.sigmoid((logit.float() + bias).transpose(1, 2))
        return (x if ok is None else torch.where(ok, x, pad)).contiguous()

    beta = gates(s["beta_logit"], s["beta_bias"], 1.0)
    gate = None
    if s["gate_logit"] is not None:
        gate = gates(s["gate_logit"], s["gate_bias"], 0.0)
    elif ok is not None:
        gate = ok.expand(beta.shape).float().contiguous()
    return {"q": rows(s["q"], True, 1), "k": rows(s["k"], True, rep), "v": rows(s["v"], False, rep),
            "beta": beta, "gate": gate}


def _block_in_grad_plain(s):
    c, dt = s["case"], s["dt"]
    B, T, H, Hk, D = c["B"], c["T"], c["H"], c["Hk"], c["D"]
    ok = _valid(s)

    def rows(x, dy, heads, unit):
        dy = dy.float().reshape(B, heads, H // heads, T, D).sum(2).permute(0, 2, 1, 3)
        if unit:
            x = x.float()
            r = torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)
            y = x * r
            dy = r * (dy - y * (y * dy).sum(-1, keepdim=True))
        if ok is not None:
            dy = torch.where(ok[:, 0, :, None, None], dy, 0.0)
        return dy.to(dt).contiguous()

    def gates(logit, bias, d):
        x = logit.float() + bias
        dx = d.transpose(1, 2) * torch.sigmoid(x) * torch.sigmoid(-x)
        if ok is not None:
            dx = torch.where(ok[:, 0, :, None], dx, 0.0)
        return dx.to(dt).contiguous(), dx.double().sum((0, 1)).float()

    out = {"dq": rows(s["q"], s["dq"], H, True), "dk": rows(s["k"], s["dk"], Hk, True),
           "dv": rows(s["v"], s["dv"], Hk, False)}
    out["dbeta_logit"], out["dbeta_bias"] = gates(s["beta_logit"], s["beta_bias"], s["dbeta"])
    if s["gate_logit"] is not None:
        out["dgate_logit"], out["dgate_bias"] = gates(s["gate_logit"], s["gate_bias"], s["dgate"])
    return out


def _chunks(x, N, C, fill=0.0):
    """[B, H, T, ...] -> [B*H, N, C, ...], padded with ``fill`` at the end."""
    B, H, T = x.shape[:3]
    x = x.reshape(B * H, T, *x.shape[3:])
    if N * C != T:
        x = torch.cat([x, x.new_full((B * H, N * C - T, *x.shape[2:]), fill)], 1)
    return x.reshape(B * H, N, C, *x.shape[2:])


def _decays(beta, C, least):
    """Cumulative log decays, in 64 bits: inside every chunk [BH, N, C], of whole chunks
    before each chunk boundary [BH, N + 1]."""
    l = torch.cumsum(torch.log(beta.double()).clamp_min(math.log(least) if least else -150.0), -1)
    L = torch.cumsum(l[..., -1], -1)
    return l, torch.cat([torch.zeros_like(L[:, :1]), L], 1)


def _carry(L, inc, first, reverse):
    """States in force at each chunk [BH, N, ...] and the one past the last of them, from the
    chunks' increments ``inc`` [BH, N, ...]; ``first`` (or None) is in force at the very start
    (``reverse``: behind the last chunk, increments being held at their chunk's start)."""
    BH, N = inc.shape[:2]
    edge, n = torch.arange(N + 1, device=inc.device)[:, None], torch.arange(N, device=inc.device)[None, :]
    if reverse:
        W = torch.where(n >= edge, torch.exp((L[:, None, :N] - L[:, :, None]).clamp_max(0.0)), 0.0)
        W0, rows, last = torch.exp(L[:, N:] - L), slice(1, None), 0
    else:
        W = torch.where(n < edge, torch.exp((L[:, :, None] - L[:, None, 1:]).clamp_max(0.0)), 0.0)
        W0, rows, last = torch.exp(L), slice(0, N), N
    S = (W.float() @ inc.reshape(BH, N, -1)).reshape(BH, N + 1, *inc.shape[2:])
    if first is not None:
        S = S + W0.float()[:, :, None, None] * first.reshape(BH, 1, *inc.shape[2:])
    return S[:, rows], S[:, last]


def _linear_parts(s, least):
    c = s["case"]
    C = min(_CHUNK, c["T"])
    N = -(-c["T"] // C)
    q, k, v = (_chunks(s[n], N, C).float() for n in ("q", "k", "v"))
    l, L = _decays(_chunks(s["beta"], N, C, 1.0), C, least)
    t = torch.arange(C, device=q.device)
    W = torch.where(t[:, None] >= t[None, :], torch.exp((l[..., :, None] - l[..., None, :]).clamp_max(0.0)),
                    0.0).float()
    g = torch.ones_like(l).float() if s["gate"] is None else _chunks(s["gate"], N, C).float()
    end = torch.exp(l[..., -1:] - l).float()
    inc = (v * (g * end)[..., None]).transpose(-1, -2) @ k
    M, last = _carry(L, inc, s["state"], False)
    return C, N, q, k, v, g, l, L, W, end, M, last


def _whole(x, case):
    """[BH, N, C, ...] -> [B, H, T, ...] without the padding."""
    B, H, T = case["B"], case["H"], case["T"]
    return x.reshape(B, H, -1, *x.shape[3:])[:, :, :T].contiguous()


def _linear_plain(s):
    C, N, q, k, v, g, l, L, W, end, M, last = _linear_parts(s, None)
    o = ((q @ k.transpose(-1, -2)) * W * g[..., None, :]) @ v
    o = o + torch.exp(l).float()[..., None] * (q @ M.transpose(-1, -2))
    c = s["case"]
    return _whole((s["scale"] * o).to(s["dt"]), c), last.reshape(c["B"], c["H"], c["D"], c["D"])


def _linear_grad_plain(s):
    c, dt, sc = s["case"], s["dt"], s["scale"]
    C, N, q, k, v, g, l, L, W, end, M, _ = _linear_parts(s, _BETA_MIN)
    do = _chunks(s["dout"], N, C).float()
    b = torch.exp(l).float()
    E, first = _carry(L, (do * (sc * b)[..., None]).transpose(-1, -2) @ q, s["dfinal"], True)
    S = (q @ k.transpose(-1, -2)) * W * sc
    P = (do @ v.transpose(-1, -2)) * W * sc
    dq_state = sc * b[..., None] * (do @ M)
    dv_state = end[..., None] * (k @ E.transpose(-1, -2))
    dk_state = end[..., None] * (v @ E)
    dq = dq_state + (P * g[..., None, :]) @ k
    dv = dv_state + S.transpose(-1, -2) @ do
    dk = dk_state + P.transpose(-1, -2) @ q
    # what passes through beta_t: every (write before t, read at or after t)
    pair = S * (do @ v.transpose(-1, -2))                       # [s, i], without the gate
    eta = (v * dv_state).sum(-1)
    dgate = eta + pair.sum(-2)
    t = torch.arange(C, device=q.device)
    before = torch.where(t[:, None] < t[None, :], 1.0, 0.0)     # [i, t]: i < t
    inside = ((pair * g[..., None, :]) @ before * (t[:, None] >= t[None, :])).sum(-2)
    zeta = (q * dq_state).sum(-1)
    through = torch.exp(l[..., -1]).float()[..., None] * (E * M).sum((-1, -2))[..., None]
    after = zeta.flip(-1).cumsum(-1).flip(-1)
    early = ((g * eta)[..., None, :] @ before)[..., 0, :]
    beta = _chunks(s["beta"], N, C, 1.0).clamp_min(_BETA_MIN)
    dbeta = (through + after + early + inside) / beta
    out = {"dq": _whole(dq.to(dt), c), "dk": _whole((g[..., None] * dk).to(dt), c),
           "dv": _whole((g[..., None] * dv).to(dt), c), "dbeta": _whole(dbeta, c)}
    if s["gate"] is not None:
        out["dgate"] = _whole(dgate, c)
    if s["state"] is not None:
        out["dstate"] = first.reshape(c["B"], c["H"], c["D"], c["D"])
    return out


def _linear_step_plain(s):
    M, k, v = s["state"], s["k"].float(), s["v"].float()
    if s["gate"] is not None:
        v = v * s["gate"][..., None]
    M.mul_(s["beta"][..., None, None]).add_(v[..., :, None] * k[..., None, :])
    return (s["scale"] * (M @ s["q"].float()[..., None])[..., 0]).to(s["dt"]), M


def _out_parts(s):
    u = s["o"].float()
    if s["skip"] is not None:
        u = u + s["skip"][:, None, None] * s["v"].float()
    r = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
    z = s["z"].float().permute(0, 2, 1, 3) if s["z"] is not None else None
    return u, r, z


def _block_out_plain(s):
    u, r, z = _out_parts(s)
    y = u * r * s["w"]
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return y.permute(0, 2, 1, 3).to(s["dt"]).contiguous()


def _block_out_grad_plain(s):
    u, r, z = _out_parts(s)
    dt, dy, n = s["dt"], s["dy"].float().permute(0, 2, 1, 3), u * r
    out = {}
    if z is not None:
        sg = torch.sigmoid(z)
        out["dz"] = (dy * n * s["w"] * sg * (1 + z * torch.sigmoid(-z))).to(dt).permute(0, 2, 1, 3).contiguous()
        dy = dy * z * sg
    out["dw"] = (dy * n).double().sum((0, 1, 2)).float()
    dn = dy * s["w"]
    du = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    out["do"] = du.to(dt)
    if s["skip"] is not None:
        out["dv"] = (s["skip"][:, None, None] * du).to(dt)
        out["dskip"] = (du * s["v"].float()).double().sum((0, 2, 3)).float()
    return out


_PLAIN = {"block_in": _block_in_plain, "block_in_grad": _block_in_grad_plain,
          "linear": _linear_plain, "linear_grad": _linear_grad_plain,
          "linear_step": _linear_step_plain, "block_out": _block_out_plain,
          "block_out_grad": _block_out_grad_plain}


# --------------------------------------------------------------------------
# The framework's calls
# --------------------------------------------------------------------------
def _run_own(s):
    from test_ridge_regression_b200 import gka

    op = s["case"]["op"]
    if op == "block_in":
        q, k, v, beta, gate = gka.gka_block_in(
            s["q"], s["k"], s["v"], s["beta_logit"], gate_logit=s["gate_logit"],
            beta_bias=s["beta_bias"], gate_bias=s["gate_bias"], lengths=s["lengths"], eps=EPS)
        return {"q": q, "k": k, "v": v, "beta": beta, "gate": gate}
    if op == "block_in_grad":
        return gka.gka_block_in_backward(
            s["q"], s["k"], s["beta_logit"], s["dq"], s["dk"], s["dv"], s["dbeta"],
            gate_logit=s["gate_logit"], dgate=s["dgate"], beta_bias=s["beta_bias"],
            gate_bias=s["gate_bias"], lengths=s["lengths"], eps=EPS)
    if op == "linear":
        last = torch.empty(*s["q"].shape[:2], s["q"].shape[3], s["q"].shape[3], device=s["q"].device)
        o = gka.gka_linear_forward(s["q"], s["k"], s["v"], s["beta"], gate=s["gate"], scale=s["scale"],
                                   initial_state=s["state"], final_state=last)
        return o, last
    if op == "linear_grad":
        return gka.gka_linear_backward(s["q"], s["k"], s["v"], s["beta"], s["dout"], gate=s["gate"],
                                       scale=s["scale"], initial_state=s["state"],
                                       dfinal_state=s["dfinal"])
    if op == "linear_step":
        o = gka.gka_linear_decode_step(s["state"], s["q"], s["k"], s["v"], s["beta"], gate=s["gate"],
                                       scale=s["scale"])
        return o, s["state"]
    if op == "block_out":
        return gka.gka_block_out(s["o"], s["w"], z=s["z"], v=s["v"], skip=s["skip"], eps=EPS)
    return gka.gka_block_out_backward(s["o"], s["w"], s["dy"], z=s["z"], v=s["v"], skip=s["skip"], eps=EPS)


def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op, D, B, H, T = case["op"], case["D"], case["B"], case["H"], case["T"]
    es = 2 if case["dtype"] == "bf16" else 4
    n = B * H * T
    if op.startswith("block_in"):
        raw, gates = B * T * (H + 2 * case["Hk"]) * D * es, 2 if case["gate"] else 1
        # the gradient reads the raw q, k and the incoming dq, dk, dv and writes as much as q, k, v
        if op == "block_in":
            return {"bytes": raw + 3 * n * D * es + n * gates * (es + 4), "flops": 10 * n * D}
        kin = B * T * (H + case["Hk"]) * D * es
        return {"bytes": kin + raw + 3 * n * D * es + n * gates * (2 * es + 4), "flops": 24 * n * D}
    if op.startswith("linear"):
        state = B * H * D * D * 4
        gate = 4 if case["gate"] else 0
        if op == "linear_step":
            return {"bytes": 2 * state + n * (4 * D * es + 4 + gate), "flops": 5 * n * D * D}
        if op == "linear":
            return {"bytes": n * (4 * D * es + 4 + gate) + state * (2 if case["state"] else 1),
                    "flops": 4 * n * D * D}
        return {"bytes": n * (7 * D * es + 8 + 2 * gate) + state * (3 if case["state"] else 0),
                "flops": 12 * n * D * D}
    rows = 2 + (1 if case["z"] else 0) + (1 if case["skip"] else 0)
    if op == "block_out":
        return {"bytes": rows * n * D * es, "flops": 12 * n * D}
    # o, dy (z, v) read; do (dz, dv) written
    return {"bytes": (3 + (2 if case["z"] else 0) + (2 if case["skip"] else 0)) * n * D * es,
            "flops": 30 * n * D}


# --------------------------------------------------------------------------
# The definitions in 64 bits: token by token, gradients by the adjoint recurrence
# or by differentiating the definition
# --------------------------------------------------------------------------
def _exact_block_in(q, k, v, bl, gl, bb, gb, lengths, H):
    rep = H // k.shape[2]
    qh = q / torch.sqrt(q.pow(2).sum(-1, keepdim=True) + EPS)
    kh = k / torch.sqrt(k.pow(2).sum(-1, keepdim=True) + EPS)
    kh, vh = (torch.stack([x] * rep, 3).flatten(2, 3) for x in (kh, v))
    beta = 1 / (1 + torch.exp(-(bl + bb)))
    gate = 1 / (1 + torch.exp(-(gl + gb))) if gl is not None else None
    if lengths is not None:
        pad = torch.arange(q.shape[1], device=q.device).unsqueeze(0) >= lengths.unsqueeze(1)
        qh, kh, vh = (x.masked_fill(pad[:, :, None, None], 0.0) for x in (qh, kh, vh))
        beta = beta.masked_fill(pad[:, :, None], 1.0)
        gate = (torch.ones_like(beta) if gate is None else gate).masked_fill(pad[:, :, None], 0.0)
    return [x.transpose(1, 2) if x is not None else None for x in (qh, kh, vh, beta, gate)]


def _exact_block_out(o, w, z, v, skip):
    u = o if skip is None else o + v * skip.view(1, -1, 1, 1)
    y = w * u / torch.sqrt(u.pow(2).mean(-1, keepdim=True) + EPS)
    y = y.transpose(1, 2)
    return y if z is None else y * (z / (1 + torch.exp(-z)))


def _exact_linear(s, keep):
    """Token by token; with ``keep`` the states before every keep-th token."""
    q, k, v, beta = (s[n].double() for n in ("q", "k", "v", "beta"))
    g = s["gate"].double() if s["gate"] is not None else torch.ones_like(beta)
    B, H, T, D = q.shape
    M = s["state"].double().clone() if s["state"] is not None else q.new_zeros(B, H, D, D)
    gv = v * g[..., None]
    o, kept = torch.empty_like(q), []
    for t in range(T):
        if keep and t % keep == 0:
            kept.append(M.clone())
        M.mul_(beta[:, :, t, None, None]).addcmul_(gv[:, :, t, :, None], k[:, :, t, None, :])
        if not keep:
            torch.matmul(M, q[:, :, t, :, None], out=o[:, :, t, :, None])
    return o * s["scale"], M, kept, (q, k, v, beta, g, gv)


def _exact_linear_grad(s):
    keep = 64
    _, _, kept, (q, k, v, beta, g, gv) = _exact_linear(s, keep)
    B, H, T, D = q.shape
    do = s["dout"].double() * s["scale"]
    R = s["dfinal"].double().clone() if s["dfinal"] is not None else q.new_zeros(B, H, D, D)
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    dbeta = torch.empty_like(beta)
    Ms = q.new_empty(keep + 1, B, H, D, D)
    for n in range(len(kept) - 1, -1, -1):
        t0, t1 = n * keep, min(T, (n + 1) * keep)
        Ms[0] = kept[n]
        for t in range(t0, t1):
            torch.mul(Ms[t - t0], beta[:, :, t, None, None], out=Ms[t - t0 + 1])
            Ms[t - t0 + 1].addcmul_(gv[:, :, t, :, None], k[:, :, t, None, :])
        for t in range(t1 - 1, t0 - 1, -1):
            R.addcmul_(do[:, :, t, :, None], q[:, :, t, None, :])
            torch.matmul(do[:, :, t, None, :], Ms[t - t0 + 1], out=dq[:, :, t, None, :])
            torch.matmul(v[:, :, t, None, :], R, out=dk[:, :, t, None, :])
            torch.matmul(R, k[:, :, t, :, None], out=dv[:, :, t, :, None])
            dbeta[:, :, t] = (R * Ms[t - t0]).sum((-1, -2))
            R.mul_(beta[:, :, t, None, None])
    out = {"dq": dq, "dk": dk * g[..., None], "dv": dv * g[..., None], "dbeta": dbeta}
    if s["gate"] is not None:
        out["dgate"] = (dv * v).sum(-1)
    if s["state"] is not None:
        out["dstate"] = R
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = lambda n: s[n].double() if s[n] is not None else None  # noqa: E731
    if op == "linear":
        o, M, _, _ = _exact_linear(s, 0)
        return o, M
    if op == "linear_grad":
        return _exact_linear_grad(s) if case["T"] <= 32768 else None
    if op == "linear_step":
        M, k, v = f64("state"), f64("k"), f64("v")
        g = f64("gate") if s["gate"] is not None else torch.ones_like(f64("beta"))
        M = torch.einsum("bh,bhij->bhij", f64("beta"), M) + torch.einsum("bh,bhi,bhj->bhij", g, v, k)
        return s["scale"] * torch.einsum("bhij,bhj->bhi", M, f64("q")), M
    names = (["q", "k", "v", "beta_logit", "gate_logit", "beta_bias", "gate_bias"]
             if op.startswith("block_in") else ["o", "w", "z", "v", "skip"])
    leaves = {n: f64(n).detach().requires_grad_() if s[n] is not None else None for n in names}
    if op.startswith("block_in"):
        out = _exact_block_in(*leaves.values(), s["lengths"], case["H"])
        if op == "block_in":
            return dict(zip(("q", "k", "v", "beta", "gate"), [x.detach() if x is not None else None for x in out]))
        ups = [f64(n) for n in ("dq", "dk", "dv", "dbeta", "dgate")]
        names = {"q": "dq", "k": "dk", "v": "dv", "beta_logit": "dbeta_logit", "gate_logit": "dgate_logit",
                 "beta_bias": "dbeta_bias", "gate_bias": "dgate_bias"}
    else:
        out = [_exact_block_out(*leaves.values())]
        if op == "block_out":
            return out[0].detach()
        ups = [f64("dy")]
        names = {"o": "do", "w": "dw", "z": "dz", "v": "dv", "skip": "dskip"}
    loss = sum((x * d).sum() for x, d in zip(out, ups) if d is not None)
    used = [n for n in names if leaves[n] is not None]
    return {names[n]: x for n, x in zip(used, torch.autograd.grad(loss, [leaves[n] for n in used]))}
