"""bf16 inputs, elements for themselves: outputs and gradients that are small beside the terms they
are sums of are as near as their own rounding, like those of fp32 arithmetic on the same inputs."""
import pytest
import torch

from linear_ref import linear, linear_grad, linear_inputs
from test_ridge_regression_b200 import build, gka

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8   # half a step of bf16, relative to the value


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def near(got, want, terms, share):
    """|got - want| within the rounding of the result and `share` of the terms' sizes."""
    return ((got.double() - want).abs() <= HALF * want.abs() + share * terms).all()


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 130, 1500])
def test_little_of_a_large_state(D, T):
    """A state whose first two columns (rows) differ by 2^-10 of them, read by e0 - e1: what a query
    reads that the rest of the memory is orthogonal to.  The first of T tokens has all of it (the
    others write nothing; beta is 1).  The state's parts leave 2^-25 of it, and each of their three
    products is off by at most 2^-23 of its largest term: 2^-21 of the terms in all."""
    gen = torch.Generator().manual_seed(61)
    B, H = 2, 9
    S = torch.randn(B, H, D, D, generator=gen)
    S[..., 1] = S[..., 0] * (1 + 2.0 ** -10 * torch.randn(B, H, D, generator=gen))
    R = S.transpose(-1, -2).contiguous()   # dk reads rows of the state's gradient, and dq of the state
    S, R = S.cuda(), R.cuda()
    pair, zero = (torch.zeros(B, H, T, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    pair[..., 0], pair[..., 1] = 1.0, -1.0
    one = torch.ones(B, H, T, device="cuda")
    o = gka.gka_linear_forward(pair, zero, zero, one, initial_state=S)
    want = (S[..., 0].double() - S[..., 1].double())[:, :, None].expand(B, H, T, D)
    terms = (S[..., 0].abs() + S[..., 1].abs()).double()[:, :, None]
    assert near(o, want, terms, 2.0 ** -21)
    g = gka.gka_linear_backward(zero, zero, zero, one, pair, initial_state=R)
    assert near(g["dq"], want, terms, 2.0 ** -21)
    for n, a, X in (("dv", (zero, pair, zero), S), ("dk", (zero, zero, pair), R)):
        g = gka.gka_linear_backward(*a, one, zero, dfinal_state=X)
        assert near(g[n], want, terms, 2.0 ** -21), n


def erasing(D, T, resets):
    """Unit key e0, written with V and, one token on, with -V: what later tokens read of the pair is
    2^-12 of either, by the decay between the two.  64 heads, the pair at another place in each.
    Returns (rows e0 at the pair, rows +-V at the pair, rows e0 everywhere, the decays)."""
    gen = torch.Generator().manual_seed(62 + T)
    B, H = 2, 32
    unit, value, read = (torch.zeros(B * H, T, D) for _ in range(3))
    read[..., 0] = 1.0
    for h in range(B * H):
        i = 4 + (h * 29) % min(T - 6, 200)
        unit[h, i:i + 2, 0] = 1.0
        value[h, i] = torch.randn(D, generator=gen)
        value[h, i + 1] = -value[h, i]
    beta = 1 - 2.0 ** -12 * torch.rand(B * H, T, generator=gen)
    beta[:, list(resets)] = 0.0
    rows = [x.view(B, H, T, D).bfloat16().cuda() for x in (unit, value, read)]
    return (*rows, beta.view(B, H, T).cuda())


def check_erased(D, T, resets):
    """Share: a weight's exponential is off by 2^-22, its parts by 2^-25, and the two terms' sum by
    2^-23 of them, in the chunk and again in the state: below 2^-20 in all.  The gradients let 2^-60
    of what was written pass a reset (their contract), where the definition has 0 and no terms: of
    the pair's two terms at most 2 * 2^-60 of the largest value."""
    unit, value, read, beta = erasing(D, T, resets)
    share = 2.0 ** -20
    o = gka.gka_linear_forward(read, unit, value, beta)
    assert near(o, linear(read, unit, value, beta)[0], linear(read, unit, value.abs(), beta)[0], share)
    # time reversed: two reads of opposite sign behind every write
    back = [x.flip(2) for x in (unit, value, read)]
    beta = beta.flip(2).contiguous()
    cases = {"dq": (value * 0, value, unit, read), "dv": (back[0], back[2], value * 0, back[1]),
             "dk": (back[1], value * 0, back[2], back[0])}   # q, k, v, dout
    for n, (q, k, v, do) in cases.items():
        b = beta if n != "dq" else beta.flip(2).contiguous()
        got = gka.gka_linear_backward(q, k, v, b, do)[n]
        want = linear_grad(q, k, v, b, do)[n]
        terms = linear_grad(q.abs(), k.abs(), v.abs(), b, do.abs())[n]
        passed = 2 * 2.0 ** -60 * value.double().abs().max() if resets else 0.0
        assert near(got, want, terms + passed / share, share), n


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [40, 128, 300])
def test_a_write_that_the_next_one_erases(D, T):
    check_erased(D, T, ())


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T,resets", [(40, (3,)), (128, (0, 1, 2, 3)), (300, tuple(range(4)) + tuple(range(128, 132)))])
def test_decays_keep_their_bits_behind_resets(D, T, resets):
    """A reset is the largest decay that is told apart: sums of decays behind it still hold those
    between two tokens to fp32's bits."""
    check_erased(D, T, resets)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T,gate,state", [(1, False, True), (37, True, False), (129, False, False), (400, True, True)])
def test_every_element(D, T, gate, state):
    """Random inputs, packed documents.  Share: two exponentials (2^-21), three parts (2^-25), 24
    steps of the tensor cores' sum, each off by at most 2^-23 of the terms (2^-18.4), the state's
    sum over four chunks (2^-21): below 2^-17."""
    a, kw, gen = linear_inputs(2, 3, T, D, torch.bfloat16, 71 + T, gate=gate, state=state, resets=(5, 64, 300))
    share, sc, g, S = 2.0 ** -17, kw["scale"], kw.get("gate"), kw.get("state")
    o = gka.gka_linear_forward(*a.values(), gate=g, scale=sc, initial_state=S)
    sizes = [x.abs() for x in a.values()]
    up = None if S is None else S.abs()
    assert near(o, linear(*a.values(), g, sc, S)[0], linear(*sizes, g, sc, up)[0], share)
    do = torch.randn(a["q"].shape, generator=gen).bfloat16().cuda()
    got = gka.gka_linear_backward(*a.values(), do, gate=g, scale=sc, initial_state=S, dfinal_state=S)
    want = linear_grad(*a.values(), do, g, sc, S, S)
    terms = linear_grad(*sizes, do.abs(), g, sc, up, up)
    # 2^-60 of what was written passes a reset
    written = 2.0 ** -60 * sum(float(x.double().abs().sum()) for x in (*a.values(), do))
    for n in ("dq", "dk", "dv"):
        assert near(got[n], want[n], terms[n] + written / share, share), n
