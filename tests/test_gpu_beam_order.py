"""The order of a beam selection among beams that fp32 sums of exponentials cannot tell apart."""
import math

import pytest
import torch

import ops_plain as P
import ssm_token_mixer_b200 as ia
from gpu_common import device

pytestmark = pytest.mark.gpu


def check(logits, scores, K, **kw):
    r = ia.beam_select(logits, scores, K, **kw)
    ia.check_device_errors()
    s, p, t = P.beam_select(logits, scores, K, kw.get("finished"), kw.get("end_token", 0))
    assert torch.equal(r["parents"].cpu(), p)
    assert torch.equal(r["tokens"].cpu(), t)
    # the fp32 sums of exponentials are off by at most 2e-6 (see the kernel), then one rounding
    assert ((r["scores"].cpu().double() - s).abs() <= 2e-6 + P.U * s.abs()).all()


def rows(G, V, dt, seed, duplicates):
    """One random row per request; with duplicates its largest value stands at four places."""
    x = torch.randn(G, V, generator=torch.Generator().manual_seed(seed)) * 2.5
    x = x.to(dt)
    if duplicates:
        top = x.float().max(1).values.to(dt)
        for at in (V // 7, V // 3, V - 2):
            x[:, at] = top
    return x


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1001, 4096, 33001, 50257])
@pytest.mark.parametrize("W,K", [(2, 1), (3, 1), (4, 2), (4, 4), (5, 3), (6, 6), (7, 2), (8, 1), (8, 5), (8, 7)])
@pytest.mark.parametrize("duplicates", [False, True])
def test_equal_beams(dt, V, W, K, duplicates):
    """Equal rows at equal scores: every row's sum is formed from another offset, and all of them tie."""
    device()
    G = 12
    x = rows(G, V, dt, seed=V + W, duplicates=duplicates)[:, None].expand(G, W, V).contiguous().cuda()
    check(x, torch.full((G, W), -12.5, device="cuda"), K)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1001, 33001])
@pytest.mark.parametrize("W,K", [(3, 1), (5, 2), (6, 5), (8, 3)])
def test_beams_closer_than_the_sums(dt, V, W, K):
    """Equal rows whose beams' scores are one fp32 step apart (9.5e-7, less than the sums' bound), in mixed order."""
    device()
    G = 12
    x = rows(G, V, dt, seed=V + K, duplicates=False)[:, None].expand(G, W, V).contiguous().cuda()
    gen = torch.Generator().manual_seed(W)
    step = torch.stack([torch.randperm(W, generator=gen) for _ in range(G)]).float()
    check(x, (-12.5 - step * 2.0 ** -20).cuda(), K)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W,K", [(3, 1), (4, 2), (8, 3)])
def test_the_tie_behind_a_better_beam(dt, W, K):
    """Beam 0 takes the first places by far, the others tie for the last one; a finished beam ties with its score alone."""
    device()
    G, V = 8, 7001
    x = rows(G, V, dt, seed=K, duplicates=True)[:, None].expand(G, W, V).contiguous()
    s = torch.full((G, W), -12.5)
    s[:, 0] = -2.0
    if K > 1:
        x[:, 0] = x[:, 0].float().clamp(max=1.0).to(dt)
        x[:, 0, 5] = 30.0          # one candidate of beam 0 above everything, its next ones below the others'
        s[:, 0] = -12.5
    check(x.cuda(), s.cuda(), K)
    fin = torch.zeros(G, W, dtype=torch.bool)
    fin[:, W - 1] = True
    check(x.cuda(), s.cuda(), K, finished=fin.cuda(), end_token=3)


def test_all_equal_rows_in_several_spans():
    """One value everywhere: the best places tie within a beam, so the other beams' places lie far down the list."""
    device()
    for V in (40001, 100003):
        for W, K in ((2, 1), (3, 2), (2, 8), (5, 4)):
            check(torch.full((1, W, V), 0.25, device="cuda"), torch.full((1, W), -1.0, device="cuda"), K)


@pytest.mark.parametrize("K", [1, 2, 3, 4, 6])
def test_logits_that_differ_below_a_sum(K):
    """Within a beam the scores differ exactly as the logits do, also where beam score + logit rounds to one number."""
    device()
    V = 5000
    x = torch.full((1, 2, V), -5.0, device="cuda")
    x[0, :, 7] = 1e-30
    x[0, :, 4000] = 3e-30
    x[0, :, 100] = 0.0
    x[0, 0, 4500] = 2e-30
    s = torch.tensor([[-3.0, -9.0]], device="cuda")
    r = ia.beam_select(x, s, K)
    ia.check_device_errors()
    want = [(0, 4000), (0, 4500), (0, 7), (0, 100), (0, 0), (0, 1)][:K]
    assert list(zip(r["parents"][0].tolist(), r["tokens"][0].tolist())) == want


def test_the_longest_vocabulary():
    """V = 2^31 - 1: the fp64 sums of two equal beams run to the last index that an int holds, and no further."""
    device()
    V = 2**31 - 1
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 10 * 2**30:
        pytest.skip("not enough free memory")
    x = torch.zeros(1, 2, V, dtype=torch.bfloat16, device="cuda")
    x[0, :, 5] = x[0, :, V - 1] = 12.0
    r = ia.beam_select(x, torch.full((1, 2), -1.0, device="cuda"), 3)
    ia.check_device_errors()
    assert r["parents"].tolist() == [[0, 0, 1]] and r["tokens"].tolist() == [[5, V - 1, 5]]
    want = -1.0 + 12.0 - math.log(V - 2 + 2 * math.exp(12.0))
    assert (r["scores"].cpu().double() - want).abs().max() <= 1e-9 + P.U * abs(want)   # fp64 sums, rounded once
