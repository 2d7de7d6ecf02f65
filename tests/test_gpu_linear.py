"""Gated linear recurrence (gka_linear_forward, gka_linear_backward,
gka_linear_decode_step) against its 64-bit definition, token by token, on every
type, head size and chunk edge, with resets, gates and carried states; and what a
caller may do with it: streams, graphs, aliases, determinism, offsets past 2^31."""
import pytest
import torch

from linear_ref import TOL, TOL16, TOL32, linear, linear_grad, linear_inputs, rel
from test_ridge_regression_b200 import build, gka

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def run_forward(a, kw, want_last=True, **more):
    B, H, T, D = a["q"].shape
    last = torch.full((B, H, D, D), float("nan"), device="cuda") if want_last else None
    o = gka.gka_linear_forward(a["q"], a["k"], a["v"], a["beta"], gate=kw.get("gate"), scale=kw["scale"],
                               initial_state=kw.get("state"), final_state=last, **more)
    return o, last


def run_backward(a, kw, dout, dfinal=None, **more):
    return gka.gka_linear_backward(a["q"], a["k"], a["v"], a["beta"], dout, gate=kw.get("gate"),
                                   scale=kw["scale"], initial_state=kw.get("state"), dfinal_state=dfinal,
                                   **more)


def check_forward(a, kw):
    o, last = run_forward(a, kw)
    assert gka.device_status() == 0
    ro, rM = linear(**a, **kw)
    assert rel(o, ro) <= TOL[a["q"].dtype]
    assert rel(last, rM[-1]) <= TOL32


def check_backward(a, kw, gen, with_final):
    B, H, T, D = a["q"].shape
    dout = torch.randn(B, H, T, D, generator=gen).to(a["q"].dtype).cuda()
    dfinal = torch.randn(B, H, D, D, generator=gen).cuda() if with_final else None
    got = run_backward(a, kw, dout, dfinal)
    assert gka.device_status() == 0
    want = linear_grad(a["q"], a["k"], a["v"], a["beta"], dout, kw.get("gate"), kw["scale"],
                       kw.get("state"), dfinal)
    assert got.keys() == want.keys()
    for n in want:
        err = rel(got[n], want[n])
        assert err <= TOL[got[n].dtype], (n, err)


LENGTHS = [1, 2, 31, 32, 33, 127, 128, 129, 257, 500]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", LENGTHS)
def test_forward(dtype, D, T):
    a, kw, _ = linear_inputs(2, 3, T, D, dtype, 100 + T, gate=T % 2 == 1, state=T % 3 != 0,
                             resets=(0, 5, 32, 127, 128, 300))
    check_forward(a, kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", LENGTHS)
def test_backward(dtype, D, T):
    a, kw, gen = linear_inputs(2, 3, T, D, dtype, 200 + T, gate=T % 2 == 1, state=T % 3 != 0,
                               resets=(0, 5, 32, 127, 128, 300))
    check_backward(a, kw, gen, with_final=T % 4 != 0)


@pytest.mark.parametrize("B,H,T", [(1, 1, 5000), (3, 25, 700), (2, 90, 260)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_few_and_many_heads(B, H, T, dtype):
    """One head in many segments, some, and more heads than run at a time."""
    a, kw, gen = linear_inputs(B, H, T, 128, dtype, 7, gate=True, state=True, resets=(T // 3, T - 1))
    check_forward(a, kw)
    if T < 1000:
        check_backward(a, kw, gen, True)


@pytest.mark.parametrize("D,B,H,T", [(64, 1, 1, 5000), (32, 1, 2, 1500), (32, 3, 50, 700), (64, 2, 200, 260)])
def test_narrow_heads_in_segments_and_waves(D, B, H, T):
    """bf16 heads of fewer columns than a tensor-core tile has."""
    a, kw, gen = linear_inputs(B, H, T, D, torch.bfloat16, 8, gate=True, state=True, resets=(T // 3, T - 1))
    check_forward(a, kw)
    if T < 2000:
        check_backward(a, kw, gen, True)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 200])
def test_scores_are_not_rounded_to_the_inputs_type(D, T):
    """A score of 1 + 2^-8, halfway between two bf16 values, on v = 1 - 2^-8: the product 1 - 2^-16
    rounds to 1, a rounded score's would be v or v (1 + 2^-7).  Every token is its own document."""
    q, k = (torch.zeros(1, 2, T, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q[..., 0], q[..., 1], k[..., :2] = 1.0, 2.0 ** -8, 1.0
    v = torch.full_like(q, 1 - 2.0 ** -8)
    o = gka.gka_linear_forward(q, k, v, torch.zeros(1, 2, T, device="cuda"))
    assert torch.equal(o, torch.ones_like(o))


@pytest.mark.parametrize("D", [32, 64, 128])
def test_fp32_gradients_of_bf16_inputs_read_all_of_the_state(D):
    """dgate of one token is v^T R k with R = dfinal_state: a state whose third bf16 part is as large
    as it can be (1 + 2^-9 + 2^-16 1.49, where two parts are 2^-17 off) and rows of one sign.
    24 accumulations of the tensor cores, each off by at most 2^-23 of the sum."""
    gen = torch.Generator().manual_seed(21)
    q, k, v, do = ((torch.rand(2, 3, 1, D, generator=gen) + 0.5).bfloat16().cuda() for _ in range(4))
    beta, gate = torch.ones(2, 3, 1, device="cuda"), torch.full((2, 3, 1), 0.5, device="cuda")
    R = torch.full((2, 3, D, D), 1 + 2.0 ** -9 + 1.49 * 2.0 ** -16, device="cuda")
    got = gka.gka_linear_backward(q, k, v, beta, do, gate=gate, scale=0.0, dfinal_state=R)
    want = torch.einsum("bhti,bhij,bhtj->bht", v.double(), R.double(), k.double())
    assert rel(got["dgate"], want) <= 24 * 2.0 ** -23


@pytest.mark.parametrize("T", [200, 3000])
def test_backward_long_one_head(T):
    a, kw, gen = linear_inputs(1, 2, T, 128, torch.bfloat16, 11, gate=True, state=True,
                               resets=(T // 2, T // 2 + 1))
    check_backward(a, kw, gen, True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strong_forgetting(dtype):
    """beta near 0.05: decays over a chunk far below the fp32 range."""
    a, kw, gen = linear_inputs(2, 2, 300, 128, dtype, 3, gate=True, state=True, mu=-3.0, sigma=1.0)
    check_forward(a, kw)
    check_backward(a, kw, gen, True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_forgetting_and_all_resets(dtype):
    a, kw, gen = linear_inputs(1, 2, 260, 128, dtype, 4, state=True)
    for value in (1.0, 0.0):
        a["beta"].fill_(value)
        check_forward(a, kw)
        check_backward(a, kw, gen, True)


@pytest.mark.parametrize("dtype,D", [(torch.float32, 64), (torch.bfloat16, 128)])
def test_nothing_passes_a_reset(dtype, D):
    """Outputs from a reset on do not depend, to the bit, on what came before it."""
    a, kw, _ = linear_inputs(1, 2, 400, D, dtype, 5, state=True, resets=(150,))
    o1, l1 = run_forward(a, kw)
    a["v"][:, :, :150] *= -3.0
    kw["state"] = kw["state"] * 100.0
    o2, l2 = run_forward(a, kw)
    assert torch.equal(o1[:, :, 150:], o2[:, :, 150:]) and torch.equal(l1, l2)
    assert not torch.equal(o1[:, :, :150], o2[:, :, :150])


@pytest.mark.parametrize("dtype,D", [(torch.float32, 32), (torch.bfloat16, 128)])
def test_closed_gates_keep_the_state(dtype, D):
    """gate = 0 everywhere with beta = 1: the state passes unchanged, the outputs read it."""
    a, kw, _ = linear_inputs(2, 2, 150, D, dtype, 6, gate=True, state=True)
    a["beta"].fill_(1.0)
    kw["gate"].zero_()
    o, last = run_forward(a, kw)
    assert torch.equal(last, kw["state"])
    assert rel(o, kw["scale"] * torch.einsum("bhij,bhtj->bhti", kw["state"].double(), a["q"].double())) \
        <= TOL[dtype]
    del kw["state"]
    o, last = run_forward(a, kw)
    assert not o.any() and not last.any()


def test_empty():
    a, kw, _ = linear_inputs(2, 3, 4, 64, torch.float32, 8, state=True)
    e = {n: x[:, :, :0].contiguous() for n, x in a.items()}
    o, last = run_forward(e, kw)
    assert o.shape == (2, 3, 0, 64) and torch.equal(last, kw["state"])
    o, last = run_forward(e, {"scale": 1.0})
    assert not last.any()
    df = torch.randn(2, 3, 64, 64, device="cuda")
    g = run_backward(e, kw, e["v"], df)
    assert torch.equal(g["dstate"], df) and g["dbeta"].shape == (2, 3, 0)
    n = {m: x[:0].contiguous() for m, x in a.items()}
    assert run_forward(n, {"scale": 1.0})[0].shape == (0, 3, 4, 64)


@pytest.mark.parametrize("dtype,D,H", [(torch.float32, 64, 2), (torch.bfloat16, 128, 2),
                                       (torch.bfloat16, 128, 80)])
def test_state_in_place(dtype, D, H):
    """final_state may be initial_state's own memory."""
    a, kw, _ = linear_inputs(1, H, 390, D, dtype, 9, state=True)
    o1, l1 = run_forward(a, kw)
    st = kw["state"].clone()
    o2 = gka.gka_linear_forward(a["q"], a["k"], a["v"], a["beta"], scale=kw["scale"], initial_state=st,
                                final_state=st)
    assert torch.equal(o1, o2) and torch.equal(l1, st)


@pytest.mark.parametrize("dtype,D", [(torch.float32, 64), (torch.bfloat16, 128)])
def test_sequence_in_two_calls(dtype, D):
    """A sequence cut anywhere, its state carried over, gives the whole one's outputs."""
    a, kw, _ = linear_inputs(2, 2, 333, D, dtype, 10, gate=True, state=True)
    o, last = run_forward(a, kw)
    cut = 190
    st, parts = kw["state"].clone(), []
    for sl in (slice(0, cut), slice(cut, None)):
        p = {n: x[:, :, sl].contiguous() for n, x in a.items()}
        parts.append(gka.gka_linear_forward(p["q"], p["k"], p["v"], p["beta"],
                                            gate=kw["gate"][:, :, sl].contiguous(), scale=kw["scale"],
                                            initial_state=st, final_state=st))
    assert rel(torch.cat(parts, 2), o) <= TOL[dtype] and rel(st, last) <= TOL32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("gate", [False, True])
def test_decode_steps(dtype, D, gate):
    """Steps one by one: against the definition, and as the forward's continuation."""
    a, kw, _ = linear_inputs(3, 5, 20, D, dtype, 12, gate=gate, state=True, resets=(7,))
    ro, rM = linear(**a, **kw)
    st = kw["state"].clone()
    for t in range(20):
        x = {n: y[:, :, t].contiguous() for n, y in a.items()}
        o = gka.gka_linear_decode_step(st, x["q"], x["k"], x["v"], x["beta"],
                                       gate=kw["gate"][:, :, t].contiguous() if gate else None,
                                       scale=kw["scale"])
        assert rel(o, ro[:, :, t]) <= TOL[dtype]
        assert rel(st, rM[t + 1]) <= TOL32


@pytest.mark.parametrize("dtype,D", [(torch.float32, 32), (torch.bfloat16, 128)])
def test_gradient_against_differences(dtype, D):
    """Central differences of the 64-bit loss along random directions of every input."""
    a, kw, gen = linear_inputs(1, 2, 140, D, dtype, 13, gate=True, state=True, resets=(60,))
    dout = torch.randn(a["q"].shape, generator=gen).to(dtype).cuda()
    dfinal = torch.randn(kw["state"].shape, generator=gen).cuda()
    got = run_backward(a, kw, dout, dfinal)

    def loss(x):
        o, M = linear(x["q"], x["k"], x["v"], x["beta"], x["gate"], kw["scale"], x["state"])
        return (o * dout.double()).sum() + (M[-1] * dfinal.double()).sum()

    base = {n: x.double() for n, x in {**a, "gate": kw["gate"], "state": kw["state"]}.items()}
    for n in base:
        d = torch.randn(base[n].shape, generator=gen).double().cuda()
        h = 1e-4   # the loss is linear in each of them but beta and k, whose third order is h^2
        diff = (loss({**base, n: base[n] + h * d}) - loss({**base, n: base[n] - h * d})) / (2 * h)
        g = got["d" + n].double()
        # |<g, d> - <g*, d>| <= tol |g| |d| / sqrt(numel) for independent errors; 6 of them
        lim = 6 * TOL[got["d" + n].dtype] * float(g.norm()) + 1e-6 * abs(float(diff))
        assert abs(float((g * d).sum() - diff)) <= lim, n


@pytest.mark.parametrize("dtype,D,B,H,T", [(torch.float32, 64, 2, 3, 200), (torch.bfloat16, 128, 1, 4, 900),
                                           (torch.bfloat16, 128, 2, 40, 300)])
def test_same_bits_every_time(dtype, D, B, H, T):
    a, kw, gen = linear_inputs(B, H, T, D, dtype, 14, gate=True, state=True)
    dout = torch.randn(a["q"].shape, generator=gen).to(dtype).cuda()
    o, last = run_forward(a, kw)
    g = run_backward(a, kw, dout)
    for _ in range(3):
        o2, last2 = run_forward(a, kw)
        g2 = run_backward(a, kw, dout)
        assert torch.equal(o, o2) and torch.equal(last, last2)
        assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("dtype,D", [(torch.float32, 64), (torch.bfloat16, 128)])
def test_memory_around_the_outputs_is_left_alone(dtype, D):
    """Outputs inside larger buffers, an odd length: what lies around them stays."""
    B, H, T = 1, 2, 77
    a, kw, _ = linear_inputs(B, H, T, D, dtype, 15)
    n, pad = B * H * T * D, 1024
    buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device="cuda")
    wsn = gka.linear_workspace_bytes(B, H, T, D, dtype)
    ws = torch.full((wsn + 512,), 5, dtype=torch.uint8, device="cuda")
    o = buf[pad:pad + n].view(B, H, T, D)
    gka.gka_linear_forward(a["q"], a["k"], a["v"], a["beta"], scale=kw["scale"], o=o, workspace=ws[:wsn])
    assert rel(o, linear(**a, **kw)[0]) <= TOL[dtype]
    assert (buf[:pad] == 7).all() and (buf[pad + n:] == 7).all() and (ws[wsn:] == 5).all()


def test_streams_and_graphs():
    """A side stream; two captured graphs that share one workspace, replayed in turn."""
    sets = [linear_inputs(1, 6, 700, 128, torch.bfloat16, s, gate=True, state=True) for s in (16, 17)]
    want = [run_forward(a, kw) for a, kw, _ in sets]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, last = run_forward(*sets[0][:2])
    s.synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(last, want[0][1])
    ws = torch.empty(gka.linear_workspace_bytes(1, 6, 700, 128, backward=True), dtype=torch.uint8,
                     device="cuda")
    graphs, outs, grads = [], [], []
    for a, kw, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_forward(a, kw, workspace=ws))
            grads.append(run_backward(a, kw, a["v"], workspace=ws))
        graphs.append(g)
    eager = [run_backward(a, kw, a["v"]) for a, kw, _ in sets]
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
        assert all(torch.equal(grads[i][n], eager[i][n]) for n in eager[i])


def test_offsets_past_two_to_the_31():
    """q, k, v and o of more than 2^31 elements: the last head against the same head alone."""
    H, T, D = 131, 131072, 128
    gen = torch.Generator(device="cuda").manual_seed(18)
    q, k, v = (torch.randn(1, H, T, D, generator=gen, device="cuda", dtype=torch.bfloat16) * 0.1
               for _ in range(3))
    assert q.numel() > 2 ** 31
    beta = torch.sigmoid(3 + torch.randn(1, H, T, generator=gen, device="cuda"))
    last = torch.empty(1, H, D, D, device="cuda")
    o = gka.gka_linear_forward(q, k, v, beta, final_state=last)
    for h in (0, H - 1):
        one = [x[:, h:h + 1].contiguous() for x in (q, k, v, beta)]
        l1 = torch.empty(1, 1, D, D, device="cuda")
        o1 = gka.gka_linear_forward(*one, final_state=l1)
        # the head alone runs in segments: the same up to fp32 order, then one rounding
        assert rel(o[:, h, -4096:], o1[:, 0, -4096:]) <= TOL16
        assert rel(last[:, h], l1[:, 0]) <= TOL32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [40, 900])
def test_gradients_of_a_result_that_is_still_being_written(dtype, T):
    """dout is the output of the call just before: no kernel of the gradients may read it early."""
    a, kw, _ = linear_inputs(1, 2, T, 64, dtype, 31)
    a = list(a.values())
    for _ in range(20):
        o = torch.empty_like(a[0]).fill_(float("nan"))
        torch.cuda.synchronize()
        gka.gka_linear_forward(*a, scale=kw["scale"], o=o)
        got = gka.gka_linear_backward(*a, o, scale=kw["scale"])
        torch.cuda.synchronize()
        want = gka.gka_linear_backward(*a, o, scale=kw["scale"])
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_two_streams_at_once():
    """Independent calls in flight together, each with its own workspace."""
    sets = [linear_inputs(1, 3 + 40 * (i % 2), 600 + i, 128, torch.bfloat16, 20 + i, gate=True, state=True)
            for i in range(4)]
    want = [(run_forward(a, kw), run_backward(a, kw, a["v"])) for a, kw, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for s, (a, kw, _) in zip(streams, sets):
        with torch.cuda.stream(s):
            got.append((run_forward(a, kw), run_backward(a, kw, a["v"])))
    torch.cuda.synchronize()
    assert gka.device_status() == 0
    for ((o, l), g), ((ro, rl), rg) in zip(got, want):
        assert torch.equal(o, ro) and torch.equal(l, rl)
        assert all(torch.equal(g[n], rg[n]) for n in rg)


def test_stream_argument():
    """With `stream` given, what the call allocates is that stream's: a workspace that is freed while
    the call runs goes to no other stream's work."""
    a, kw, _ = linear_inputs(2, 4, 700, 128, torch.bfloat16, 41)
    a = list(a.values())
    want = gka.gka_linear_backward(*a, a[2], scale=kw["scale"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [gka.gka_linear_backward(*a, a[2], scale=kw["scale"], stream=s) for _ in range(2)]
    n = gka.linear_workspace_bytes(2, 4, 700, 128, backward=True)
    for _ in range(4):   # the freed workspace's size, written on the current stream meanwhile
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(g[m], want[m]) for m in want)


def test_nan_decay_shows():
    """A NaN among the decays is not taken for a reset."""
    for dtype, D in ((torch.float32, 64), (torch.bfloat16, 128)):
        a, kw, _ = linear_inputs(1, 2, 200, D, dtype, 24)
        a["beta"][0, 1, 50] = float("nan")
        o, last = run_forward(a, kw)
        assert torch.isfinite(o[0, 0]).all() and torch.isfinite(last[0, 0]).all()
        assert torch.isnan(last[0, 1]).any() and torch.isnan(o[0, 1, 51:]).any()


def test_refusals():
    """What the binding does not take, with nothing launched or written."""
    a, kw, _ = linear_inputs(1, 2, 40, 64, torch.float32, 25, gate=True, state=True)
    q, k, v, b = (a[n] for n in ("q", "k", "v", "beta"))
    bad = [dict(q=q[..., ::2]), dict(k=k.half()), dict(beta=b.double()), dict(beta=b[:, :, 1:]),
           dict(v=v.cpu()), dict(q=q.transpose(1, 2))]
    for kw2 in bad:
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            gka.gka_linear_forward(**{**a, **kw2})
    for kw2 in (dict(gate=kw["gate"].half()), dict(initial_state=kw["state"][:, :1]),
                dict(final_state=kw["state"].bfloat16()), dict(o=v), dict(o=q[:, :, :20]),
                dict(workspace=torch.empty(0, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            gka.gka_linear_forward(**a, **kw2)
    with pytest.raises(gka.GkaError):
        gka.gka_linear_forward(**a, scale=float("nan"))
    big, _, _ = linear_inputs(1, 1, 4000, 128, torch.bfloat16, 26)
    n = gka.linear_workspace_bytes(1, 1, 4000, 128)
    with pytest.raises(gka.GkaError):
        gka.gka_linear_forward(**big, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises((ValueError, TypeError)):
        gka.gka_linear_backward(**a, dout=v[:, :, 1:])
    with pytest.raises((ValueError, TypeError)):
        gka.gka_linear_decode_step(kw["state"], q[:, :, 0], k[:, :, 0].contiguous(),
                                   v[:, :, 0].contiguous(), b[:, :, 0].contiguous())
    x = {n: y[:, :, 0].contiguous() for n, y in a.items()}
    with pytest.raises(ValueError):
        gka.gka_linear_decode_step(kw["state"], **x, o=x["v"])


def test_states_that_overlap_are_refused():
    a, kw, _ = linear_inputs(2, 2, 9, 32, torch.float32, 42)
    both = torch.zeros(3, 2, 32, 32, device="cuda")
    with pytest.raises(ValueError):
        gka.gka_linear_forward(*a.values(), initial_state=both[:2], final_state=both[1:])
