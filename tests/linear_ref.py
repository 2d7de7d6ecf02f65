"""64-bit definitions of the gated linear recurrence and the block's row operations,
token by token and by the adjoint recurrence: what the tests hold the kernels to.

Tolerances (relative Frobenius error).  A rounding is off by at most half a step,
eps / 2 of the value (bf16 2^-8, fp32 2^-24).
  fp32 outputs: sums of up to D + 2 chunk products plus a carry of N chunks, each
      operation off by 2^-24; the errors are relative to the terms' norm, not to their
      sum.  (128 + 256 + 128) * 2^-24 = 3.1e-5 bounds the worst alignment of signs;
      TOL32 = 2e-5 is below it and above any random one.
  bf16 outputs: one rounding of the result (2^-8) and, on the tensor cores, one of each
      weighted score (2^-8 of each term, independent of the others, so 2^-8 of the
      result's norm): TOL16 = 2 * 2^-8.
"""
import torch

TOL32, TOL16 = 2e-5, 2.0 ** -7
TOL = {torch.float32: TOL32, torch.bfloat16: TOL16}


def rel(got, want):
    """Relative Frobenius error, in 64 bits; exact zeros have to be zeros."""
    g, w = got.detach().double().cpu(), want.detach().double().cpu()
    assert g.shape == w.shape, (g.shape, w.shape)
    assert torch.isfinite(g).all()
    n = float(w.norm())
    return float((g - w).norm()) / n if n else float(g.norm())


def linear(q, k, v, beta, gate=None, scale=1.0, state=None):
    """(o, states [T + 1, B, H, D, D]) with states[t] = M_{t-1}."""
    q, k, v, beta = (x.double() for x in (q, k, v, beta))
    g = torch.ones_like(beta) if gate is None else gate.double()
    B, H, T, D = q.shape
    M = q.new_zeros(B, H, D, D) if state is None else state.double()
    o, Ms = torch.zeros_like(q), [M]
    for t in range(T):
        M = beta[:, :, t, None, None] * M + (g[:, :, t, None] * v[:, :, t])[..., :, None] * k[:, :, t, None, :]
        o[:, :, t] = scale * (M @ q[:, :, t, :, None])[..., 0]
        Ms.append(M)
    return o, Ms


def linear_grad(q, k, v, beta, dout, gate=None, scale=1.0, state=None, dfinal=None):
    _, Ms = linear(q, k, v, beta, gate, scale, state)
    q, k, v, beta, do = (x.double() for x in (q, k, v, beta, dout))
    g = torch.ones_like(beta) if gate is None else gate.double()
    B, H, T, D = q.shape
    R = q.new_zeros(B, H, D, D) if dfinal is None else dfinal.double()
    dq, dk, dv = (torch.zeros_like(q) for _ in range(3))
    db, dg = torch.zeros_like(beta), torch.zeros_like(beta)
    for t in range(T - 1, -1, -1):
        R = R + scale * do[:, :, t, :, None] * q[:, :, t, None, :]
        dq[:, :, t] = scale * (do[:, :, t, None, :] @ Ms[t + 1])[..., 0, :]
        rk = (R @ k[:, :, t, :, None])[..., 0]
        dv[:, :, t] = g[:, :, t, None] * rk
        dk[:, :, t] = g[:, :, t, None] * (v[:, :, t, None, :] @ R)[..., 0, :]
        dg[:, :, t] = (v[:, :, t] * rk).sum(-1)
        db[:, :, t] = (R * Ms[t]).sum((-1, -2))
        R = beta[:, :, t, None, None] * R
    out = {"dq": dq, "dk": dk, "dv": dv, "dbeta": db}
    if gate is not None:
        out["dgate"] = dg
    if state is not None:
        out["dstate"] = R
    return out


def block_in(q, k, v, bl, gl=None, bb=None, gb=None, lengths=None, eps=1e-6):
    q, k, v, bl = (x.double() for x in (q, k, v, bl))
    B, T, H, D = q.shape
    n = H // k.shape[2]
    qh = q * (q.square().sum(-1, keepdim=True) + eps) ** -0.5
    kh = k * (k.square().sum(-1, keepdim=True) + eps) ** -0.5
    kh, vh = (x.repeat_interleave(n, 2) for x in (kh, v))
    beta = torch.sigmoid(bl if bb is None else bl + bb.double())
    gate = None
    if gl is not None:
        gate = torch.sigmoid(gl.double() if gb is None else gl.double() + gb.double())
    if lengths is not None:
        pad = torch.arange(T, device=q.device)[None, :] >= lengths[:, None]
        qh, kh, vh = (torch.where(pad[..., None, None], 0.0, x) for x in (qh, kh, vh))
        beta = torch.where(pad[..., None], 1.0, beta)
        gate = torch.where(pad[..., None], 0.0, torch.ones_like(beta) if gate is None else gate)
    return tuple(x.transpose(1, 2) if x is not None else None for x in (qh, kh, vh, beta, gate))


def block_out(o, w, z=None, v=None, skip=None, eps=1e-6):
    o, w = o.double(), w.double()
    u = o if v is None else o + skip.double()[:, None, None] * v.double()
    y = (u * (u.square().mean(-1, keepdim=True) + eps) ** -0.5 * w).transpose(1, 2)
    return y if z is None else y * torch.nn.functional.silu(z.double())


def linear_inputs(B, H, T, D, dtype, seed, *, gate=False, state=False, resets=(), mu=3.0, sigma=1.0,
                  device="cuda"):
    """Unit q, k rows, normal v, beta = sigmoid(N(mu, sigma)) with zeros at `resets`."""
    from test_ridge_regression_b200.inputs import make_gate, make_inputs
    q, k, v, beta = make_inputs(B, H, T, D, dtype, mu, sigma, seed)
    for t in resets:
        if t < T:
            beta[..., t] = 0.0
    gen = torch.Generator().manual_seed(seed + 17)
    a = {"q": q, "k": k, "v": v, "beta": beta}
    kw = {"scale": D ** -0.5}
    if gate:
        kw["gate"] = make_gate((B, H, T), seed)
        if T > 2:
            kw["gate"][..., T // 2] = 0.0
    if state:
        kw["state"] = torch.randn(B, H, D, D, generator=gen)
    a = {n: x.to(device) for n, x in a.items()}
    kw = {n: x.to(device) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    return a, kw, gen
