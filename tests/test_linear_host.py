"""Gated linear recurrence and block rows without a GPU: the definitions the GPU tests
hold the kernels to (gradients against central differences, the chunk form of dbeta
against the adjoint recurrence), and the refusals of the C ABI and of the binding."""
import math
import struct

import pytest
import torch

import linear_ref as ref


def test_gradient_definition_against_differences():
    """A bilinear loss: central differences are exact but for beta's and h^2."""
    a, kw, gen = ref.linear_inputs(1, 2, 9, 32, torch.float32, 1, gate=True, state=True, resets=(4,),
                                   device="cpu")
    dout = torch.randn(a["q"].shape, generator=gen).double()
    dfinal = torch.randn(kw["state"].shape, generator=gen).double()
    g = ref.linear_grad(a["q"], a["k"], a["v"], a["beta"], dout, kw["gate"], kw["scale"], kw["state"], dfinal)
    base = {n: x.double() for n, x in {**a, "gate": kw["gate"], "state": kw["state"]}.items()}

    def loss(x):
        o, M = ref.linear(x["q"], x["k"], x["v"], x["beta"], x["gate"], kw["scale"], x["state"])
        return (o * dout).sum() + (M[-1] * dfinal).sum()

    for n in base:
        d = torch.randn(base[n].shape, generator=gen).double()
        h = 1e-5
        diff = (loss({**base, n: base[n] + h * d}) - loss({**base, n: base[n] - h * d})) / (2 * h)
        assert abs(float((g["d" + n] * d).sum() - diff)) <= 1e-7 * (1 + abs(float(diff))), n


@pytest.mark.parametrize("C", [8, 16])
def test_chunk_form_of_dbeta(C):
    """beta_t dbeta_t = F + sum_{s>=t} zeta_s + sum_{i<t} g_i eta_i + sum_{i<t<=s} A_si, with
    decays clamped at 2^-60, against <R_t, M_{t-1}> at resets, runs of them and tiny decays."""
    a, kw, gen = ref.linear_inputs(1, 2, 48, 32, torch.float32, 2, gate=True, state=True,
                                   resets=(0, 8, 9, 20, 47), device="cpu")
    a["beta"][..., 30] = 1e-25
    dout = torch.randn(a["q"].shape, generator=gen)
    dfinal = torch.randn(kw["state"].shape, generator=gen)
    want = ref.linear_grad(a["q"], a["k"], a["v"], a["beta"], dout, kw["gate"], kw["scale"], kw["state"], dfinal)
    q, k, v, do, g = (x.double() for x in (a["q"], a["k"], a["v"], dout, kw["gate"]))
    beta, c = a["beta"].double().clamp_min(2.0 ** -60), kw["scale"]
    T = q.shape[2]
    _, Ms = ref.linear(q, k, v, beta, g, c, kw["state"])
    E = [None] * (T // C + 1)
    E[-1] = R = dfinal.double()
    for t in range(T - 1, -1, -1):
        R = beta[:, :, t, None, None] * (R + c * do[:, :, t, :, None] * q[:, :, t, None, :])
        if t % C == 0:
            E[t // C] = R
    for n in range(T // C):
        sl = slice(n * C, (n + 1) * C)
        l = beta[:, :, sl].log().cumsum(-1)
        S, En, M = l[..., -1:], E[n + 1], Ms[n * C]
        zeta = c * l.exp() * torch.einsum("bhtv,bhvk,bhtk->bht", do[:, :, sl], M, q[:, :, sl])
        eta = (S - l).exp() * torch.einsum("bhtv,bhvk,bhtk->bht", v[:, :, sl], En, k[:, :, sl])
        w = torch.tril((l[..., :, None] - l[..., None, :]).exp())
        pair = c * w * (q[:, :, sl] @ k[:, :, sl].transpose(-1, -2)) * (do[:, :, sl] @ v[:, :, sl].transpose(-1, -2))
        assert ref.rel(eta + pair.sum(-2), want["dgate"][:, :, sl]) < 1e-12
        F = S[..., 0].exp() * (En * M).sum((-1, -2))
        A = pair * g[:, :, None, sl]
        for t in range(C):
            d = F + zeta[..., t:].sum(-1) + (g[:, :, sl] * eta)[..., :t].sum(-1) + A[..., t:, :t].sum((-1, -2))
            x, y = d / beta[:, :, n * C + t], want["dbeta"][:, :, n * C + t]
            assert ((x - y).abs() <= 1e-10 * (1 + y.abs())).all(), (n, t)


@pytest.fixture(scope="module")
def lib():
    from test_ridge_regression_b200 import build, gka
    build.build()
    return gka


OK, INVALID, UNSUPPORTED, SMALL, MISALIGNED = 0, -1, -2, -4, -7
P, ODD = 1 << 20, (1 << 20) + 4   # never dereferenced: every call here is refused first


def lin(gka, **kw):
    a = dict(q=P, k=P, v=P, beta=P, gate=None, o=P, B=1, H=2, T=8, D=64, dt=0, scale=1.0, init=None,
             last=None, ws=P, n=1 << 40)
    a.update(kw)
    return gka.lib().gka_linear_forward(a["q"], a["k"], a["v"], a["beta"], a["gate"], a["o"], a["B"], a["H"],
                                        a["T"], a["D"], a["dt"], a["scale"], a["init"], a["last"], a["ws"],
                                        a["n"], None)


def test_linear_forward_refusals(lib):
    for n in ("q", "k", "v", "beta", "o"):
        assert lin(lib, **{n: None}) == INVALID
        assert lin(lib, **{n: ODD}) == MISALIGNED
    for n in ("gate", "init", "last"):
        assert lin(lib, **{n: ODD}) == MISALIGNED
    for n in ("B", "H", "T"):
        assert lin(lib, **{n: -1}) == INVALID
    for x in (math.inf, math.nan):
        assert lin(lib, scale=x) == INVALID
    assert lin(lib, dt=2) == INVALID
    assert lin(lib, D=96) == UNSUPPORTED and lin(lib, H=70000) == UNSUPPORTED
    big = dict(T=4096, D=128, dt=1)
    assert lib.lib().gka_linear_forward_workspace_bytes(1, 2, 4096, 128, 1) > 0
    assert lin(lib, **big, n=16) == SMALL
    assert lin(lib, **big, ws=None) == INVALID and lin(lib, **big, ws=P + 16) == MISALIGNED
    assert lin(lib, B=0) == OK and lin(lib, H=0, q=None) == OK


def test_linear_backward_refusals(lib):
    def call(**kw):
        a = dict(q=P, k=P, v=P, beta=P, gate=None, dout=P, init=None, dlast=None, dq=P, dk=P, dv=P, dbeta=P,
                 dgate=None, dinit=None, B=1, H=2, T=8, D=64, dt=0, scale=1.0, ws=P, n=1 << 40)
        a.update(kw)
        return lib.lib().gka_linear_backward(*a.values(), None)

    for n in ("q", "k", "v", "beta", "dout", "dq", "dk", "dv", "dbeta", "ws"):
        assert call(**{n: None}) == INVALID, n
        assert call(**{n: ODD}) == MISALIGNED, n
    for n in ("init", "dlast", "dinit"):
        assert call(**{n: ODD}) == MISALIGNED
    assert call(gate=P) == INVALID and call(dgate=P) == INVALID
    assert call(dlast=P, dinit=P) == INVALID   # one is read while the other is written
    assert call(n=0) == SMALL and call(scale=math.nan) == INVALID
    assert call(D=16) == UNSUPPORTED and call(B=-1) == INVALID and call(B=0) == OK


def test_linear_step_refusals(lib):
    def call(**kw):
        a = dict(state=P, q=P, k=P, v=P, beta=P, gate=None, o=P, B=1, H=2, D=64, dt=1, scale=1.0)
        a.update(kw)
        return lib.lib().gka_linear_decode_step(*a.values(), None)

    for n in ("state", "q", "k", "v", "beta", "o"):
        assert call(**{n: None}) == INVALID
        assert call(**{n: ODD}) == MISALIGNED
    assert call(gate=ODD) == MISALIGNED and call(D=48) == UNSUPPORTED and call(dt=7) == INVALID
    assert call(H=-1) == INVALID and call(scale=math.inf) == INVALID and call(B=0) == OK
    assert call(B=1 << 20, H=1 << 10) == UNSUPPORTED


def rows(gka, ptr=P, sb=64 * 64, st=64, sh=64):
    return struct.pack("Pqqq", ptr or 0, sb, st, sh)


def test_block_in_refusals(lib):
    def call(**kw):
        a = dict(q=rows(lib), k=rows(lib), v=rows(lib), bl=rows(lib), gl=None, bb=None, gb=None, lengths=None,
                 qo=P, ko=P, vo=P, beta=P, gate=None, B=1, T=8, H=4, Hk=2, D=64, dt=1, eps=1e-6)
        a.update(kw)
        return lib.lib().gka_block_in_forward(*a.values(), None)

    for n in ("q", "k", "v", "bl", "qo", "ko", "vo", "beta"):
        assert call(**{n: None}) == INVALID, n
    for n in ("q", "k", "v"):
        assert call(**{n: rows(lib, None)}) == INVALID
        assert call(**{n: rows(lib, ODD)}) == MISALIGNED
        for s in ("sb", "st", "sh"):
            assert call(**{n: rows(lib, **{s: 12})}) == MISALIGNED
    for n in ("qo", "ko", "vo", "beta"):
        assert call(**{n: ODD}) == MISALIGNED
    assert call(gl=rows(lib)) == INVALID        # a gate to read, none to write
    assert call(lengths=P) == INVALID
    assert call(gate=P) == INVALID              # a gate to write, none to read
    assert call(Hk=3) == INVALID and call(Hk=0) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=math.nan) == INVALID
    assert call(D=40) == UNSUPPORTED and call(T=-1) == INVALID and call(dt=3) == INVALID
    assert call(T=0) == OK


def test_block_in_backward_refusals(lib):
    def call(**kw):
        a = dict(q=rows(lib), k=rows(lib), bl=rows(lib), gl=None, bb=None, gb=None, lengths=None, dqo=P, dko=P,
                 dvo=P, dbeta=P, dgate=None, dq=P, dk=P, dv=P, dbl=P, dgl=None, dbb=None, dgb=None, B=1, T=8,
                 H=4, Hk=2, D=64, dt=1, eps=1e-6, ws=P, n=1 << 40)
        a.update(kw)
        return lib.lib().gka_block_in_backward(*a.values(), None)

    for n in ("q", "k", "bl", "dqo", "dko", "dvo", "dbeta", "dq", "dk", "dv", "dbl", "ws"):
        assert call(**{n: None}) == INVALID, n
    for n in ("dqo", "dko", "dvo", "dbeta", "dq", "dk", "dv", "dbl", "ws"):
        assert call(**{n: ODD}) == MISALIGNED, n
    for kw in (dict(gl=rows(lib)), dict(dgate=P), dict(dgl=P), dict(dgb=P), dict(gl=rows(lib), dgate=P)):
        assert call(**kw) == INVALID, kw
    assert call(n=0) == SMALL


def test_block_out_refusals(lib):
    def fwd(**kw):
        a = dict(o=P, v=None, z=None, w=P, skip=None, y=P, B=1, T=8, H=4, D=64, dt=1, eps=1e-6)
        a.update(kw)
        return lib.lib().gka_block_out_forward(*a.values(), None)

    def bwd(**kw):
        a = dict(o=P, v=None, z=None, w=P, skip=None, dy=P, do=P, dv=None, dz=None, dw=P, dskip=None, B=1, T=8,
                 H=4, D=64, dt=1, eps=1e-6, ws=P, n=1 << 40)
        a.update(kw)
        return lib.lib().gka_block_out_backward(*a.values(), None)

    for n in ("o", "w", "y"):
        assert fwd(**{n: None}) == INVALID and fwd(**{n: ODD}) == MISALIGNED
    assert fwd(v=P) == INVALID and fwd(skip=P) == INVALID and fwd(z=rows(lib, ODD)) == MISALIGNED
    assert fwd(z=rows(lib, st=4)) == MISALIGNED and fwd(eps=math.inf) == INVALID and fwd(D=8) == UNSUPPORTED
    for n in ("o", "w", "dy", "do", "dw", "ws"):
        assert bwd(**{n: None}) == INVALID, n
    for n in ("o", "w", "dy", "do", "ws"):
        assert bwd(**{n: ODD}) == MISALIGNED, n
    for kw in (dict(v=P, skip=P), dict(z=rows(lib)), dict(dz=P), dict(dv=P), dict(dskip=P)):
        assert bwd(**kw) == INVALID, kw
    assert bwd(n=0) == SMALL


def test_binding_refuses_host_tensors(lib):
    a, kw, _ = ref.linear_inputs(1, 1, 4, 32, torch.float32, 3, device="cpu")
    with pytest.raises(ValueError):
        lib.gka_linear_forward(**a)
    with pytest.raises(ValueError):
        lib.gka_linear_backward(**a, dout=a["v"])
    x = torch.zeros(1, 4, 1, 32)
    with pytest.raises(ValueError):
        lib.gka_block_in(x, x, x, x[..., 0])
    with pytest.raises(ValueError):
        lib.gka_block_out(x, torch.ones(32))


def test_workspace_queries(lib):
    f, b = lib.lib().gka_linear_forward_workspace_bytes, lib.lib().gka_linear_backward_workspace_bytes
    for dt in (0, 1):
        for D in (32, 64, 128):
            for T in (0, 1, 100, 4096):
                assert f(2, 3, T, D, dt) % 256 == 0 and b(2, 3, T, D, dt) % 256 == 0
                assert b(2, 3, T, D, dt) >= f(2, 3, T, D, dt)
    assert f(1, 1, 64, 100, 0) == 0 and b(-1, 1, 64, 64, 0) == 0
    assert lib.lib().gka_block_out_backward_workspace_bytes(2, 9, 3, 64, 1) >= 4 * (64 + 1) * 3
    assert lib.lib().gka_block_in_backward_workspace_bytes(2, 9, 4, 3, 64, 1) == 0
