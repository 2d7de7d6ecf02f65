"""Edges of the block's row operations: no eps under the root, an output over the gate's rows,
no query heads, far negative gates."""
import pytest
import torch

import linear_ref as ref
from linear_ref import TOL32, rel
from test_gpu_block_rows import make_in, make_out
from test_ridge_regression_b200 import build, gka

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_block_in_without_eps(dtype, D):
    """eps = 0: padding is zero rows and zero gradients, as with any eps."""
    args, kw, g = make_in(3, 37, 4, 2, D, dtype, 31, lengths=[37, 0, 13])
    got = gka.gka_block_in(*args, **kw, eps=0.0)
    want = ref.block_in(*args, kw["gate_logit"], kw["beta_bias"], kw["gate_bias"], kw["lengths"], 0.0)
    for x, y in zip(got, want):
        tol = 2.0 ** -8 + 1e-6 if x.dtype == torch.bfloat16 else 1e-6   # half a step of the type
        assert rel(x, y) <= tol
    for x in got[:3]:
        assert not x[1].any() and not x[2, :, 13:].any()
    ups = [torch.randn(3, 4, 37, D, generator=g).to(dtype).cuda() for _ in range(3)]
    ups += [torch.randn(3, 4, 37, generator=g).cuda() for _ in range(2)]
    back = gka.gka_block_in_backward(args[0], args[1], args[3], *ups[:4], dgate=ups[4], **kw, eps=0.0)
    leaves = [x.double().requires_grad_() for x in args[:3]]
    out = ref.block_in(*leaves, args[3], kw["gate_logit"], kw["beta_bias"], kw["gate_bias"], None, 0.0)
    real = torch.arange(37, device="cuda")[None, :] < kw["lengths"][:, None]
    loss = sum((torch.where(real[:, None, :, None], x, 0.0) * u.double()).sum() for x, u in zip(out, ups[:3]))
    for n, y in zip(("dq", "dk", "dv"), torch.autograd.grad(loss, leaves)):
        assert rel(back[n], y) <= (2.0 ** -8 if dtype == torch.bfloat16 else TOL32), n
        assert not back[n][1].any() and not back[n][2, 13:].any(), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 7, 250])
def test_block_out_gradient_without_eps(dtype, D, T):
    """eps = 0 and real rows that are not zero: lanes past a block's run add nothing to dw and dskip."""
    o, w, kw, g = make_out(1, T, 3, D, dtype, 32, True, True)
    dy = torch.randn(1, T, 3, D, generator=g).to(dtype).cuda()
    got = gka.gka_block_out_backward(o, w, dy, **kw, eps=0.0)
    leaves = {n: x.double().requires_grad_() for n, x in {"o": o, "w": w, **kw}.items()}
    loss = (ref.block_out(**leaves, eps=0.0) * dy.double()).sum()
    for n, y in zip(leaves, torch.autograd.grad(loss, list(leaves.values()))):
        x = got["d" + n]
        assert rel(x, y) <= (TOL32 if x.dtype == torch.float32 else 2.0 ** -8), n


def test_an_output_over_the_gate_is_refused():
    """y in z's memory, all of it, a part, or between z's strided rows: other blocks still read z."""
    o, w, _, _ = make_out(2, 8, 4, 64, torch.bfloat16, 33, False, False)
    rows = torch.zeros(3, 8, 4, 64, device="cuda", dtype=torch.bfloat16)
    for z, y in ((rows[:2], rows[:2]), (rows[:2], rows[1:])):
        with pytest.raises(ValueError):
            gka.gka_block_out(o, w, z=z, y=y)
    wide = torch.zeros(2, 8, 12, 64, device="cuda", dtype=torch.bfloat16)
    inside = wide.view(-1)[4 * 64:4 * 64 + o.numel()].view(2, 8, 4, 64)
    with pytest.raises(ValueError):
        gka.gka_block_out(o, w, z=wide[:, :, :4], y=inside)
    y = gka.gka_block_out(o, w, z=rows[:2], y=rows[2:].new_zeros(2, 8, 4, 64))   # apart: taken
    assert not y.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_query_heads(dtype):
    """H = 0: the gradients of the key and value heads are empty sums, written as such."""
    q, bl = torch.zeros(2, 5, 0, 64, device="cuda", dtype=dtype), torch.zeros(2, 5, 0, device="cuda", dtype=dtype)
    k = torch.ones(2, 5, 3, 64, device="cuda", dtype=dtype)
    up, db = q.transpose(1, 2).contiguous(), torch.zeros(2, 0, 5, device="cuda")
    assert gka.gka_block_in(q, k, k, bl)[1].shape == (2, 0, 5, 64)
    for _ in range(3):   # the allocator hands out memory that held NaN
        dirty = [torch.full_like(k, float("nan")) for _ in range(4)]
        torch.cuda.synchronize()
        del dirty
        got = gka.gka_block_in_backward(q, k, bl, up, up, up, db)
        assert not got["dk"].any() and not got["dv"].any() and got["dq"].shape == q.shape


def test_far_gates_element_by_element():
    """z from -95 to 40 in bf16, each element for itself.  The result's rounding (2^-8), at most
    2^-15 of arithmetic (the exponential's error grows with |z|, to 2^-16 at -90), and half of
    bf16's smallest step, 2^-134, with the same again for an exponential below fp32's normals."""
    D, T = 128, 64
    g = torch.Generator().manual_seed(34)
    o = torch.randn(1, 1, T, D, generator=g).bfloat16().cuda()
    o = torch.where(o.abs() < 0.1, torch.ones_like(o), o)
    z = torch.linspace(-95.0, 40.0, T * D).view(1, T, 1, D).bfloat16().cuda()
    z = torch.where((z + 1.2785).abs() < 0.5, torch.full_like(z, 2.0), z)   # silu' has its zero there
    w = torch.rand(D, generator=g).cuda() + 0.5
    dy = (torch.rand(1, T, 1, D, generator=g) + 0.5).bfloat16().cuda()
    want = ref.block_out(o, w, z=z)
    y = gka.gka_block_out(o, w, z=z).double()
    leaf = z.double().requires_grad_()
    (dz,) = torch.autograd.grad((ref.block_out(o, w, z=leaf) * dy.double()).sum(), leaf)
    got = gka.gka_block_out_backward(o, w, dy, z=z)["dz"].double()
    for x, e in ((y, want), (got, dz)):
        assert ((x - e).abs() <= (2.0 ** -8 + 2.0 ** -15) * e.abs() + 2.0 ** -133).all()
    assert (y[z < -80].abs() > 0).any()
