"""The state of linear attention: fp32 accuracy of what the sequence calls return and of what many steps of decoding keep.

U = 2^-24 is half an fp32 step.  Tokens are few here and the rest zero, so that a state's roundings can be counted."""
import math

import numpy as np
import pytest
import torch

import ops_plain as P
import ssm_token_mixer_b200 as ia
from gpu_common import device

pytestmark = pytest.mark.gpu
U = P.U


def sparse(N, at, dk, dv, seed):
    """q, k, v [1,2,N,.] with tokens at the given places only."""
    gen = torch.Generator().manual_seed(seed)
    q, k, v = (torch.zeros(1, 2, N, d) for d in (dk, dk, dv))
    for t in at:
        q[:, :, t], k[:, :, t], v[:, :, t] = (torch.randn(1, 2, d, generator=gen) for d in (dk, dk, dv))
    return [x.bfloat16().cuda() for x in (q, k, v)]


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("N,at", [(2, (0, 1)), (7, (0, 3, 6)), (128, (2, 60, 125)), (300, (5, 130, 290)), (900, (100, 520, 890))])
@pytest.mark.parametrize("segments", [1, 2, 4])
def test_returned_state(dk, dv, N, at, segments, monkeypatch):
    """The weighted values of a returned state enter its product in three bf16 parts, which leave 2^-24 of a value; with
    two, 2^-16 would be left, several times this bound."""
    device()
    monkeypatch.setenv("IA_LINEAR_SEGMENTS", str(segments))
    q, k, v = sparse(N, at, dk, dv, seed=N + dk)
    g = torch.tensor([-0.003, -0.011]).cuda()
    assert ia.linear_path(1, 2, N, dk, dv, "bf16") == "tensor_core"
    got = ia.linear_prefill_fwd(q, k, v, g, want_state=True)["state"].view(2, dk, dv).double()
    ia.check_device_errors()
    want, bound = torch.zeros_like(got), torch.zeros_like(got)
    chunks = -(-N // 128)
    for t in at:
        for h in range(2):
            far = N - 1 - t
            term = math.exp(float(g[h]) * far) * torch.outer(k[0, h, t].double(), v[0, h, t].double())
            want[h] += term
            # the weight (expf's 2 ulp and its argument's rounding), its product, what three parts leave; three
            # accumulations of at most two steps each, the parts' sum; per chunk the decay's 2 ulp, its product and a sum
            n = 4 + abs(float(g[h])) * far + 1 + 1 + 3 * 2 * 2 + 1 + 6 * chunks
            bound[h] += n * U * term.abs()
    assert bound.max() <= 40 * U * want.abs().max() * 3 + 1e-30
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{((got - want).abs() / bound.clamp(min=1e-30)).max().item():.2f} times the bound"


@pytest.mark.parametrize("dt,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 64), (torch.float32, 40)])
@pytest.mark.parametrize("decay,N", [(x, n) for x in (-1e-3, -0.04, -0.3, -0.69, -0.7, -2.5, -9.0) for n in (1, 2, 9, 33, 150, 400)
                                     if x * n > -80])                 # above fp32's range
@pytest.mark.parametrize("segments", [1, 3])
def test_a_state_that_only_decays(dt, d, decay, N, segments, monkeypatch):
    """Keys of zero (padding): the state after them is lambda^N times the one before, to fp32, however small that is."""
    device()
    monkeypatch.setenv("IA_LINEAR_SEGMENTS", str(segments))
    gen = torch.Generator().manual_seed(N)
    q, k, v = torch.zeros(1, 1, N, d), torch.zeros(1, 1, N, d), torch.randn(1, 1, N, d, generator=gen)
    s = torch.randn(1, 1, d, d, generator=gen).cuda()
    g = torch.tensor([decay]).cuda()
    args = [x.to(dt).cuda() for x in (q, k, v)]
    got = ia.linear_prefill_fwd(*args, g, state_in=s, want_state=True)["state"].view(d, d).double()
    ia.check_device_errors()
    exact = float(g[0].double())
    want = math.exp(exact * N) * s.view(d, d).double()
    # per chunk (32 tokens at least): the decay's 2 ulp (4 U, and as much again where it is taken from 1), a product and
    # a sum; the exponents' roundings add up to |g| N U
    n = (-(-N // 32)) * 8 + abs(exact) * N + 8
    assert ((got - want).abs() <= n * U * want.abs()).all(), ((got / want - 1).abs().max() / U).item()
    # and token by token
    state = s.flatten().clone()
    x = [a[:, :, 0].contiguous() for a in args]
    for _ in range(N):
        ia.linear_decode_step(*x, g, state)
    ia.check_device_errors()
    n = N * 8 + abs(exact) * N + 8
    assert ((state.view(d, d).double() - want).abs() <= n * U * want.abs()).all()


def test_decode_does_not_drift():
    """4096 steps whose decay lies midway between two fp32 numbers: its rounding would shift every entry the same way.

    Rounded to fp32, such a decay is off by 2^-25, and 4096 steps by 1.2e-4.  What remains is rounded once a step, which
    as a random walk is sqrt(4096) U = 3.8e-6 per entry and vanishes in the mean over 8192 entries, and the 2 ulp of
    expm1 at 2^-11, which add up to 4096 * 2^-34 = 2.4e-7."""
    device()
    T, d = 4096, 64
    g = -np.float32(2.0) ** -11 * (1 + np.arange(4096, dtype=np.float32) * np.float32(2.0) ** -20)
    exact = np.exp(g.astype(np.float64))
    off = (exact.astype(np.float32).astype(np.float64) - exact) / exact
    g = torch.tensor([g[off.argmax()], g[off.argmin()]]).cuda()
    assert off.max() > 2.9e-8 and off.min() < -2.9e-8
    gen = torch.Generator().manual_seed(1)
    s = torch.randn(1, 2, d, d, generator=gen).cuda()
    z = torch.zeros(1, 2, d, dtype=torch.bfloat16, device="cuda")
    state = s.flatten().clone()
    for _ in range(T):
        ia.linear_decode_step(z, z, z, g, state)
    ia.check_device_errors()
    want = torch.exp(g.double() * T)[None, :, None, None] * s.double()
    rel = (state.view_as(s).double() / want - 1)[0]
    assert rel.mean((1, 2)).abs().max() <= 1e-6
    assert rel.abs().max() <= 6 * math.sqrt(T) * U
