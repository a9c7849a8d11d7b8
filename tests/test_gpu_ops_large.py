"""Offsets past 32 bits: the last rows of tensors with more than 2^31 elements."""
import pytest
import torch

import ops_plain as P
import ssm_token_mixer_b200 as ia
from gpu_common import device

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def room(gigabytes):
    device()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 2**30:
        pytest.skip("not enough free memory")


def test_linear_prefill():
    room(24)
    B, H, N, d = 513, 64, 1024, 64
    assert B * H * N * d > 2**31
    q = torch.zeros(B, H, N, d, dtype=BF, device="cuda")
    k, v = torch.zeros_like(q), torch.zeros_like(q)
    for x in (q, k, v):
        x[-1].normal_()
    g = torch.full((H,), -0.05, device="cuda")
    r = ia.linear_prefill_fwd(q, k, v, g, want_state=True)
    ia.check_device_errors()
    o, bo, S, bS = P.linear_bounds(q[-1:], k[-1:], v[-1:], g, d ** -0.5, True)
    assert ((r["o"][-1:].double() - o).abs() <= bo).all()
    assert ((r["state"].view(B, H, d, d)[-1:].double() - S).abs() <= bS).all()
    assert r["o"][-2].abs().max() == 0


def test_decode_and_reorder():
    room(40)
    B, H, d = 8196, 16, 128
    assert B * H * d * d > 2**31
    q, k, v = (torch.randn(B, H, d, device="cuda").to(BF) for _ in range(3))
    g = torch.full((H,), -0.1, device="cuda")
    state = torch.zeros(B * H * d * d, device="cuda")
    last = state.view(B, H, d, d)[-4:].normal_()
    parents = torch.zeros(B // 4, 4, dtype=torch.int32, device="cuda")
    parents[-1] = torch.tensor([3, 0, -1, 1])
    moved = ia.linear_state_reorder(state, parents, B, H, d, d).view(B, H, d, d)
    want = torch.stack([last[3], last[0], torch.zeros_like(last[0]), last[1]])
    assert torch.equal(moved[-4:], want)
    del moved
    before = last.double()
    o = ia.linear_decode_step(q, k, v, g, state)["o"]
    ia.check_device_errors()
    lam = torch.exp(g.double())[None, :, None, None]
    S = lam * before + k[-4:].double()[..., :, None] * v[-4:].double()[..., None, :]
    w = (q[-4:].double()[..., None, :] @ S)[..., 0, :] * d ** -0.5
    n = (q[-4:].double().abs()[..., None, :] @ S.abs())[..., 0, :] * d ** -0.5
    # the decay's exponential (an ulp, 2 U) and a product on what was there, k v exact, one sum; then 128 terms in fp32
    # of a state that is off by this much, and the rounding of the output
    assert ((state.view(B, H, d, d)[-4:].double() - S).abs() <= 3 * P.U * before.abs() + 2 * P.U * S.abs()).all()
    assert ((o[-4:].double() - w).abs() <= 2.0 ** -8 * w.abs() + (d + 16) * P.U * n).all()


def test_layer_norm():
    room(30)
    D = 1024
    rows = 2**31 // D + 7
    x = torch.zeros(rows, D, dtype=BF, device="cuda")
    x[-5:].normal_(0.3, 2.0)
    w = torch.randn(D, device="cuda")
    r = ia.layer_norm_fwd(x, w, None)
    y, mean, rstd, _ = P.layer_norm(x[-5:], w, None, 1e-5)
    # at most 45 roundings on the way of a term: 45 U mean|x| = 4.4e-6 for the mean, 45 U + an rsqrt for rstd; with
    # |xhat|, |w| and |dy| below 5, 5 and 11 these are 6e-5 in y and 1.5e-5 in xhat, so 8e-4 in five rows' sums
    assert ((r["mean"][-5:].double() - mean).abs() <= 1e-5).all()
    assert ((r["rstd"][-5:].double() / rstd - 1).abs() <= 1e-5).all()
    assert ((r["y"][-5:].double() - y).abs() <= 2.0 ** -8 * y.abs() + 1e-4).all()
    b = ia.layer_norm_bwd(x, x, r["mean"], r["rstd"], w)   # the rows of zeros add nothing to the sums
    dx, dw, db = P.layer_norm_grads(x[-5:], x[-5:], w, 1e-5)
    assert ((b["dx"][-5:].double() - dx).abs() <= 2.0 ** -8 * dx.abs() + 1e-3).all()
    assert ((b["dweight"].double() - dw).abs() <= 1e-3).all() and ((b["dbias"].double() - db).abs() <= 1e-3).all()
    assert b["dx"][0].abs().max() == 0
    ia.check_device_errors()


def test_beam_select():
    room(12)
    G, W, V = 669, 64, 50257
    assert G * W * V > 2**31
    x = torch.zeros(G, W, V, dtype=BF, device="cuda")
    x[-1].normal_(0.0, 2.5)
    s = -torch.rand(G, W, device="cuda")
    r = ia.beam_select(x, s, 8)
    score, parent, token = P.beam_select(x[-1:], s[-1:], 8, None, 0)
    assert torch.equal(r["parents"][-1:].cpu(), parent) and torch.equal(r["tokens"][-1:].cpu(), token)
    assert ((r["scores"][-1:].cpu().double() - score).abs() <= 2e-6 + P.U * score.abs()).all()
    ia.check_device_errors()
