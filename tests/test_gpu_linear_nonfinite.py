"""Linear attention with NaN or infinities at every lane of a warp: the tokens before stay as they were, bit for bit."""
import pytest
import torch

import ssm_token_mixer_b200 as ia
from gpu_common import device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("want_state", [False, True])
@pytest.mark.parametrize("first", [0, 33, 128, 230])
def test_at_every_lane(d, want_state, first):
    """The mark of the first bad token splits a warp of output rows at any of its lanes."""
    device()
    gen = torch.Generator().manual_seed(first + d)
    N, j = 300, d // 2 + 1
    q, k, v = (torch.randn(1, 2, N, d, generator=gen).bfloat16().cuda() for _ in range(3))
    g = torch.tensor([-0.1, -0.01]).cuda()
    clean = ia.linear_prefill_fwd(q, k, v, g, want_state=want_state)
    grads = ia.linear_fwd_bwd(q, k, v, g, v)
    for u in range(first, first + 32):
        bad = v.clone()
        bad[0, 1, u, j] = float("nan") if u % 2 else float("inf")
        bad[0, 1, min(N - 1, u + 3), 0] = float("-inf")   # a second one in the same chunk, in another column
        r = ia.linear_prefill_fwd(q, k, bad, g, want_state=want_state)
        b = ia.linear_fwd_bwd(q, k, bad, g, bad)
        for o, want in ((r["o"], clean["o"]), (b["o"], grads["o"])):
            assert torch.equal(o[0, 0], want[0, 0]) and torch.equal(o[0, 1, :u], want[0, 1, :u])
            assert not torch.isfinite(o[0, 1, u:, j].float()).any()
        if want_state:
            assert torch.equal(r["state"].view(2, -1)[0], clean["state"].view(2, -1)[0])
            assert not torch.isfinite(r["state"].view(2, d, d)[1, :, j]).any()
    # towards the start, dv is the sum over the later tokens: one in dO reaches none after it
    dO = v.clone()
    for u in range(first, first + 32):
        bad = dO.clone()
        bad[0, 1, u, j] = float("nan")
        b = ia.linear_fwd_bwd(q, k, v, g, bad)
        assert torch.equal(b["dv"][0, 0], grads["dv"][0, 0]) and torch.equal(b["dv"][0, 1, u + 1:], grads["dv"][0, 1, u + 1:])
        assert not torch.isfinite(b["dv"][0, 1, :u + 1, j].float()).any()
    ia.check_device_errors()
