"""bf16 outputs of linear attention on the tensor cores: off by their own rounding, not by roundings of the operands."""
import pytest
import torch

import ops_plain as P
import ssm_token_mixer_b200 as ia
from gpu_common import device
from test_gpu_linear import make, within

pytestmark = pytest.mark.gpu


def bounds(x, y, z, g, scale, state=None, reverse=False):
    """The definition in fp64 and what the kernels may be off by.

    A term of an output is off by 2^-16 of itself from the second part of P (or of S) and by as much again from the
    second part of w z on its way through S; by the roundings in fp32 on its way (the products over dx, a chunk's sum, the
    decays: 2 ulp and an argument's rounding of exponents whose weight makes them U / 2 each, and three per chunk); and
    the sum by its rounding to bf16, 2^-8.  With P and S rounded to bf16 once, 2^-8 of the terms would be added, many
    times this where they cancel."""
    out, _ = P.recurrence(x, y, z, g, state, reverse)
    mag, _ = P.recurrence(x.abs(), y.abs(), z.abs(), g, None if state is None else state.abs(), reverse)
    n = x.shape[3] + 256 + 3 * (x.shape[2] // 128 + 1) + 16
    out, err = out * scale, (2.0 ** -15 + n * P.U) * mag * abs(scale)
    return out, err + P.BF * (out.abs() + err) + 1e-30


@pytest.mark.parametrize("shape", [(1, 2, 1, 64, 64), (2, 2, 5, 64, 64), (1, 2, 130, 64, 64), (1, 1, 300, 128, 128),
                                   (1, 2, 500, 64, 128), (2, 1, 260, 128, 64), (1, 2, 1025, 64, 64)])
@pytest.mark.parametrize("segments", [1, 3])
def test_outputs_and_gradients(shape, segments, monkeypatch):
    device()
    monkeypatch.setenv("IA_LINEAR_SEGMENTS", str(segments))
    t = make(*shape, torch.bfloat16, seed=shape[2], state=True, grad=True)
    q, k, v, dO, g = t["q"], t["k"], t["v"], t["dO"], t["g"]
    scale = shape[3] ** -0.5
    o, bo = bounds(q, k, v, g, scale, t["s"])
    for want in (False, True):
        within(ia.linear_prefill_fwd(q, k, v, g, state_in=t["s"], want_state=want)["o"], o, bo)
    r = ia.linear_fwd_bwd(q, k, v, g, dO)
    ia.check_device_errors()
    for name, (x, y, z, rev) in {"o": (q, k, v, False), "dq": (dO, v, k, False), "dk": (v, dO, q, True),
                                 "dv": (k, q, dO, True)}.items():
        want, bound = bounds(x, y, z, g, scale, reverse=rev)
        within(r[name], want, bound)
        # as norms: the rounding to bf16, and the terms' 2^-15 at most, which random signs leave far smaller
        rounding = (want.to(torch.bfloat16).double() - want).norm()
        assert (r[name].double() - want).norm() <= 1.02 * rounding + 2.0 ** -15 * want.norm()
