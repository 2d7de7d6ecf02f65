"""The block's row operations (gka_block_in, gka_block_out and their gradients) against
their 64-bit definitions and autograd through them, and the whole run they belong to:
projections -> block_in -> layer or linear recurrence -> block_out, and back."""
import pytest
import torch

import linear_ref as ref
from linear_ref import TOL, TOL16, TOL32, rel
from test_ridge_regression_b200 import build, gka

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def make_in(B, T, H, Hk, D, dtype, seed, gate=True, bias=True, lengths=None):
    """Views of one projection's output, as a program has them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, (H + 2 * Hk) * D + 2 * H, generator=g).to(dtype).cuda()
    # rows at 16-byte steps: the logits lie behind the rows in storage of their own
    qkv, ba = x[..., :(H + 2 * Hk) * D].contiguous(), x[..., (H + 2 * Hk) * D:].contiguous()
    q, k, v = qkv.split([H * D, Hk * D, Hk * D], -1)
    kw = {"gate_logit": ba[..., H:] if gate else None, "lengths": None}
    kw["beta_bias"] = (3 + torch.randn(H, generator=g)).cuda() if bias else None
    kw["gate_bias"] = torch.randn(H, generator=g).cuda() if bias and gate else None
    if lengths is not None:
        kw["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return (q.unflatten(-1, (H, D)), k.unflatten(-1, (Hk, D)), v.unflatten(-1, (Hk, D)), ba[..., :H]), kw, g


def ref_in(args, kw, eps=1e-6):
    return ref.block_in(*args, kw["gate_logit"], kw["beta_bias"], kw["gate_bias"], kw["lengths"], eps)


SHAPES = [(1, 1, 1, 1), (2, 3, 2, 1), (3, 37, 8, 2), (2, 129, 12, 12), (4, 260, 6, 3)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("gate,bias,pad", [(True, True, False), (False, False, True), (True, False, True),
                                           (False, True, False)])
def test_block_in(dtype, D, shape, gate, bias, pad):
    B, T, H, Hk = shape
    lengths = [(T * (i + 1)) // B if i else 0 for i in range(B)] if pad else None
    args, kw, _ = make_in(B, T, H, Hk, D, dtype, 1, gate, bias, lengths)
    got = gka.gka_block_in(*args, **kw)
    want = ref_in(args, kw)
    for n, x, y in zip(("q", "k", "v", "beta", "gate"), got, want):
        assert (x is None) == (y is None), n
        if x is not None:
            # one rounding of each value: half a step of its type, and fp32 arithmetic before it
            tol = 2.0 ** -8 + 1e-6 if x.dtype == torch.bfloat16 else 1e-6
            assert (x.double() - y).abs().max() <= tol * y.abs().max(), n
    if not pad:   # the values pass unchanged
        assert torch.equal(got[2], args[2].repeat_interleave(H // Hk, 2).transpose(1, 2))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("gate,bias,pad", [(True, True, False), (False, False, True), (True, True, True)])
def test_block_in_backward(dtype, D, shape, gate, bias, pad):
    B, T, H, Hk = shape
    lengths = [(T * (i + 1)) // B if i else 0 for i in range(B)] if pad else None
    args, kw, g = make_in(B, T, H, Hk, D, dtype, 2, gate, bias, lengths)
    ups = [torch.randn(B, H, T, D, generator=g).to(dtype).cuda() for _ in range(3)]
    ups += [torch.randn(B, H, T, generator=g).cuda(), torch.randn(B, H, T, generator=g).cuda() if gate else None]
    got = gka.gka_block_in_backward(args[0], args[1], args[3], *ups[:4], dgate=ups[4], **kw)
    names = ["dq", "dk", "dv", "dbeta_logit", "dgate_logit", "dbeta_bias", "dgate_bias"]
    leaves = [x.double().requires_grad_() if x is not None else None
              for x in (*args, kw["gate_logit"], kw["beta_bias"], kw["gate_bias"])]
    out = ref.block_in(*leaves[:4], leaves[4], leaves[5], leaves[6], kw["lengths"])
    loss = sum((x * u.double()).sum() for x, u in zip(out, ups) if u is not None)
    want = dict(zip([n for n, x in zip(names, leaves) if x is not None],
                    torch.autograd.grad(loss, [x for x in leaves if x is not None])))
    assert got.keys() == want.keys()
    for n in want:
        err = rel(got[n], want[n])
        # biases: a sum of B T terms of either sign, each within 2^-22, against their norm
        assert err <= (TOL32 if got[n].dtype == torch.float32 else 2.0 ** -8), (n, err)


def test_block_in_padding_is_not_read():
    """Padding may hold anything: NaN and infinities do not reach the outputs or gradients."""
    args, kw, g = make_in(3, 40, 4, 2, 64, torch.bfloat16, 3, lengths=[40, 0, 13])
    clean = gka.gka_block_in(*args, **kw)
    ups = [torch.randn(3, 4, 40, 64, generator=g).bfloat16().cuda() for _ in range(3)] + [
        torch.randn(3, 4, 40, generator=g).cuda() for _ in range(2)]

    def back():
        return gka.gka_block_in_backward(args[0], args[1], args[3], *ups[:4], dgate=ups[4], **kw)

    gclean = back()
    for x in (*args, kw["gate_logit"]):
        x[1] = float("nan")
        x[2, 13:] = float("inf")
    for u in ups:
        u[1] = float("nan")
        u[2, :, 13:] = float("-inf")
    for x, y in zip(gka.gka_block_in(*args, **kw), clean):
        assert torch.equal(x, y)
    gdirty = back()
    assert all(torch.equal(gdirty[n], gclean[n]) for n in gclean)
    q, k, v, beta, gate = clean
    assert not q[1].any() and not v[2, :, 13:].any()
    assert (beta[1] == 1).all() and not gate[1].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_in_extreme_rows(dtype):
    """Zero rows stay zero (eps), large and small rows come out as unit rows or x / sqrt(eps);
    saturated logits give 0 and 1 and no NaN gradient."""
    args, kw, _ = make_in(1, 8, 2, 2, 64, dtype, 4, bias=False)
    q, bl = args[0], args[3]
    q[0, 0], q[0, 1], q[0, 2] = 0.0, q[0, 1] * 1e15, q[0, 2] * 1e-6
    bl[0, 3], bl[0, 4] = 200.0, -200.0
    got = gka.gka_block_in(*args, **kw)
    want = ref_in(args, kw)
    assert not got[0][0, :, 0].any()
    assert rel(got[0], want[0]) <= 2.0 ** -8 and rel(got[3], want[3]) <= 1e-6
    assert (got[3][0, :, 3] == 1).all() and (got[3][0, :, 4] == 0).all()
    ups = [torch.ones_like(got[i]) for i in range(5)]
    back = gka.gka_block_in_backward(q, args[1], bl, *ups[:4], dgate=ups[4], **kw)
    assert all(torch.isfinite(x).all() for x in back.values())


def make_out(B, T, H, D, dtype, seed, z, skip):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    kw = {"z": None, "v": None, "skip": None}
    if z:   # a view between other columns
        kw["z"] = r(B, T, 3 * H * D).to(dtype).cuda()[..., H * D:2 * H * D].unflatten(-1, (H, D))
    if skip:
        kw["v"], kw["skip"] = r(B, H, T, D).to(dtype).cuda(), r(H).cuda()
    return r(B, H, T, D).to(dtype).cuda(), (1 + 0.3 * r(D)).cuda(), kw, g


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (2, 3, 5), (3, 131, 4), (1, 600, 12)])
@pytest.mark.parametrize("z,skip", [(True, True), (False, False), (True, False), (False, True)])
def test_block_out(dtype, D, B, T, H, z, skip):
    o, w, kw, g = make_out(B, T, H, D, dtype, 5, z, skip)
    y = gka.gka_block_out(o, w, **kw)
    assert rel(y, ref.block_out(o, w, **kw)) <= (2.0 ** -8 if dtype == torch.bfloat16 else 1e-6)
    dy = torch.randn(B, T, H, D, generator=g).to(dtype).cuda()
    got = gka.gka_block_out_backward(o, w, dy, **kw)
    names = {"o": o, "w": w, **{n: x for n, x in kw.items() if x is not None}}
    leaves = {n: x.double().requires_grad_() for n, x in names.items()}
    grads = torch.autograd.grad((ref.block_out(**leaves) * dy.double()).sum(), list(leaves.values()))
    want = {"d" + n: x for n, x in zip(leaves, grads)}
    assert got.keys() == want.keys()
    for n in want:
        err = rel(got[n], want[n])
        assert err <= (TOL32 if got[n].dtype == torch.float32 else 2.0 ** -8), (n, err)


def test_empty_rows():
    args, kw, _ = make_in(2, 4, 2, 1, 32, torch.float32, 6)
    cut = lambda x: x[:, :0] if x is not None and x.dim() > 2 else x  # noqa: E731
    q, k, v, beta, gate = gka.gka_block_in(*map(cut, args), **{n: cut(x) for n, x in kw.items()})
    assert q.shape == (2, 2, 0, 32) and gate.shape == (2, 2, 0)
    back = gka.gka_block_in_backward(cut(args[0]), cut(args[1]), cut(args[3]), q, k, v, beta, dgate=gate,
                                     **{n: cut(x) for n, x in kw.items()})
    assert not back["dbeta_bias"].any() and not back["dgate_bias"].any()
    o, w, kw, _ = make_out(1, 0, 3, 64, torch.bfloat16, 7, True, True)
    assert gka.gka_block_out(o, w, **kw).shape == (1, 0, 3, 64)
    g = gka.gka_block_out_backward(o, w, o.transpose(1, 2).contiguous(), **kw)
    assert not g["dw"].any() and not g["dskip"].any()


def test_same_bits_and_graphs():
    args, kw, g = make_in(3, 500, 8, 2, 128, torch.bfloat16, 8, lengths=[500, 77, 0])
    ups = [torch.randn(3, 8, 500, 128, generator=g).bfloat16().cuda() for _ in range(3)] + [
        torch.randn(3, 8, 500, generator=g).cuda() for _ in range(2)]
    o, w, okw, _ = make_out(3, 500, 8, 128, torch.bfloat16, 9, True, True)
    dy = o.transpose(1, 2).contiguous()

    def run():
        r = list(gka.gka_block_in(*args, **kw))
        r += gka.gka_block_in_backward(args[0], args[1], args[3], *ups[:4], dgate=ups[4], **kw).values()
        r.append(gka.gka_block_out(o, w, **okw))
        return r + list(gka.gka_block_out_backward(o, w, dy, **okw).values())

    first = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(first, run(), captured):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("dtype,D", [(torch.float32, 64), (torch.bfloat16, 128)])
def test_a_whole_block_and_its_gradients(dtype, D):
    """block_in -> linear recurrence -> block_out over a padded batch, and the way back,
    against 64-bit autograd of the composed definitions."""
    B, T, H, Hk = 3, 70, 4, 2
    args, kw, g = make_in(B, T, H, Hk, D, dtype, 10, lengths=[70, 41, 0])
    z = torch.randn(B, T, H, D, generator=g).to(dtype).cuda()
    w, skip = torch.rand(D, generator=g).cuda(), torch.randn(H, generator=g).cuda()
    dy = torch.randn(B, T, H, D, generator=g).to(dtype).cuda()
    sc = D ** -0.5
    q, k, v, beta, gate = gka.gka_block_in(*args, **kw)
    last = torch.empty(B, H, D, D, device="cuda")
    o = gka.gka_linear_forward(q, k, v, beta, gate=gate, scale=sc, final_state=last)
    y = gka.gka_block_out(o, w, z=z, v=v, skip=skip)
    go = gka.gka_block_out_backward(o, w, dy, z=z, v=v, skip=skip)
    gl = gka.gka_linear_backward(q, k, v, beta, go["do"], gate=gate, scale=sc)
    gi = gka.gka_block_in_backward(args[0], args[1], args[3], gl["dq"], gl["dk"], gl["dv"] + go["dv"],
                                   gl["dbeta"], dgate=gl["dgate"], **kw)
    # a sequence's state is the one after its own last token
    rq, rk, rv, rb, rg = ref_in(args, kw)
    _, Ms = ref.linear(rq, rk, rv, rb, rg, sc)
    assert rel(last[1], Ms[41][1]) <= (TOL16 if dtype == torch.bfloat16 else TOL32)
    assert not last[2].any()
    leaves = {n: x.double().requires_grad_() for n, x in zip(
        ("dq", "dk", "dv", "dbeta_logit", "dgate_logit", "dbeta_bias", "dgate_bias", "dz", "dw", "dskip"),
        (*args, kw["gate_logit"], kw["beta_bias"], kw["gate_bias"], z, w, skip))}
    L = list(leaves.values())
    xq, xk, xv, xb, xg = ref.block_in(*L[:4], L[4], L[5], L[6], kw["lengths"])
    M, os = xq.new_zeros(B, H, D, D), []
    for t in range(T):
        M = xb[:, :, t, None, None] * M + xg[:, :, t, None, None] * xv[:, :, t, :, None] * xk[:, :, t, None, :]
        os.append(sc * (M @ xq[:, :, t, :, None])[..., 0])
    ry = ref.block_out(torch.stack(os, 2), L[8], L[7], xv, L[9])
    want = dict(zip(leaves, torch.autograd.grad((ry * dy.double()).sum(), L)))
    got = {**gi, "dz": go["dz"], "dw": go["dw"], "dskip": go["dskip"]}
    # a padded token's row is zero into the norm: its gate gets no gradient and skip none
    # bf16: four roundings of intermediate rows (q, k, o, do or dq), then the result's
    tol = 5 * 2.0 ** -8 if dtype == torch.bfloat16 else 2 * TOL32
    assert rel(y, ry) <= tol
    for n in want:
        assert rel(got[n], want[n]) <= tol, (n, rel(got[n], want[n]))


def test_block_in_feeds_the_ridge_layer():
    """block_in's outputs are gka_forward_gated's inputs as they stand."""
    args, kw, _ = make_in(2, 128, 2, 1, 128, torch.bfloat16, 11)
    q, k, v, beta, gate = gka.gka_block_in(*args, **kw)
    o = gka.gka_forward_gated(q, k, v, beta, gate, 0.5, 20, 64)
    import oracle
    want = oracle.forward(q.cpu(), k.cpu(), v.cpu(), beta.cpu(), 0.5, 20, gate=gate.cpu())["o"]
    assert rel(o, torch.from_numpy(want)) <= 2e-2   # the layer's own bar for bf16
    y = gka.gka_block_out(o, torch.ones(128, device="cuda"))
    assert rel(y, ref.block_out(o, torch.ones(128, device="cuda"))) <= TOL[torch.bfloat16]


def test_refusals():
    args, kw, g = make_in(2, 8, 4, 2, 64, torch.bfloat16, 12)
    q, k, v, bl = args
    wide = torch.zeros(2, 8, 4, 128, device="cuda", dtype=torch.bfloat16)
    for bad in ((wide[..., ::2], k, v, bl), (q.float(), k, v, bl), (q, k[:, :, :1], v, bl), (q, k, v, bl[:1]),
                (q.cpu(), k, v, bl), (q, wide[:, :, :3, :64], wide[:, :, :3, :64], bl)):
        with pytest.raises((ValueError, TypeError, gka.GkaError)):
            gka.gka_block_in(*bad, gate_logit=kw["gate_logit"])
    odd = torch.zeros(2, 8, 4 * 64 + 3, device="cuda", dtype=torch.bfloat16)[..., 3:].unflatten(-1, (4, 64))
    with pytest.raises(gka.GkaError):   # rows off the 16-byte grid
        gka.gka_block_in(odd, k, v, bl)
    with pytest.raises(ValueError):
        gka.gka_block_in(*args, gate_bias=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        gka.gka_block_in(*args, lengths=torch.tensor([8, 8], device="cuda"))   # int64
    with pytest.raises(gka.GkaError):
        gka.gka_block_in(*args, eps=float("nan"))
    o, w, okw, _ = make_out(2, 8, 4, 64, torch.bfloat16, 13, True, True)
    with pytest.raises(ValueError):
        gka.gka_block_out(o, w, v=okw["v"])
    with pytest.raises(ValueError):
        gka.gka_block_out(o, w[:32])
    with pytest.raises(ValueError):
        gka.gka_block_out(o, w, y=o.view(2, 8, 4, 64))
    with pytest.raises(ValueError):
        gka.gka_block_out_backward(o, w, o)
