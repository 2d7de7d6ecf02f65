"""Operands that arrive late: every product of the tensor-core linear recurrence waits for the load
of what it reads, and no call's outputs hold what another call left in shared memory."""
import re
from pathlib import Path

import pytest
import torch

from linear_ref import TOL16, linear, linear_grad, linear_inputs, rel
from test_ridge_regression_b200 import build, gka

SOURCE = Path(build.CSRC, "linear_tc.cuh").read_text()


def part(start, end):
    i = SOURCE.index(start)
    return SOURCE[i:SOURCE.index(end, i)]


def waits_before(text, product):
    """Barriers that `text` waits on before its first `product`."""
    return set(re.findall(r"\bwait\((b_\w+)", text[:text.index(product)]))


def test_issuers_wait_for_their_operands():
    """Barriers of the loads (b_xy, b_z), or of a role that has waited for them, before each product.
    b_xfree is x's copy to TMEM, made once b_xy is there; b_parts is u z, formed from z."""
    kernel = part("k_linear_tc(const __grid_constant__", "// Segment aggregates:")
    state = kernel[kernel.index("if (warp == 16)"):kernel.index("else if (warp == 17)")]
    scores = kernel[kernel.index("else if (warp == 17)"):kernel.index("else if (warp == 18)")]
    parts = kernel[kernel.index("---- state: thread has"):]
    assert "b_xy" in waits_before(scores, "cp_128x256b(")             # x and y, before P too
    assert {"b_xfree", "b_s"} <= waits_before(state, "tmem + kOS")
    assert "b_parts" in waits_before(state, "tmem + kDS")
    assert "b_z" in waits_before(parts, "lt_parts(")
    loop = scores[scores.index("for (int it = 0;"):]
    assert {"b_z", "b_pb"} <= waits_before(loop, "tmem + kOI")
    agg = part("k_linear_agg_tc(const", "// dbeta and dgate of one 128-token chunk")
    assert "b_parts" in waits_before(agg, "mma_f16(")
    assert "b_yz" in waits_before(agg[agg.index("warp < 16"):], "lt_parts(")


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 100, 128, 300])
def test_nothing_of_another_call_is_read(D, T):
    """Calls of very large values in between, and inputs out of L2: the same bits every time."""
    a, kw, gen = linear_inputs(2, 74, T, D, torch.bfloat16, 51 + T)
    dout = torch.randn(a["q"].shape, generator=gen).bfloat16().cuda()
    huge = {n: x * 1e6 if n == "v" else x for n, x in a.items()}
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def both(x, up):
        o = gka.gka_linear_forward(**x, scale=kw["scale"])
        return {"o": o, **gka.gka_linear_backward(**x, dout=up, scale=kw["scale"])}

    first = both(a, dout)
    for _ in range(10):
        both(huge, dout * 1e6)
        flush.zero_()
        again = both(a, dout)
        assert all(torch.equal(first[n], again[n]) for n in first)
    assert gka.device_status() == 0
    few = {n: x[:1, :2].contiguous() for n, x in a.items()}
    assert rel(first["o"][:1, :2], linear(**few, scale=kw["scale"])[0]) <= TOL16
    want = linear_grad(*few.values(), dout[:1, :2], None, kw["scale"])
    for n in ("dq", "dk", "dv"):
        assert rel(first[n][:1, :2], want[n]) <= TOL16, n
