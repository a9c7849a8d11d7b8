"""Beam selection and state reordering on the GPU against their definitions."""
import pytest
import torch

import ops_plain as P
import ssm_token_mixer_b200 as ia
from gpu_common import device

pytestmark = pytest.mark.gpu
INF = float("inf")


def check(logits, scores, K, finished=None, end_token=0):
    r = ia.beam_select(logits, scores, K, finished=finished, end_token=end_token)
    ia.check_device_errors()
    s, p, t = P.beam_select(logits, scores, K, finished, end_token)
    assert torch.equal(r["parents"].cpu(), p)
    assert torch.equal(r["tokens"].cpu(), t)
    got = r["scores"].cpu().double()
    ok = torch.isfinite(s)
    assert torch.equal(got[~ok], s[~ok])
    # the fp32 sums of exponentials are off by at most 2e-6 (see the kernel), then one rounding
    assert ((got[ok] - s[ok]).abs() <= 2e-6 + P.U * s[ok].abs()).all()
    return r


def data(G, W, V, dt, seed=0, std=2.5):
    g = torch.Generator().manual_seed(seed * 7919 + V)
    return ((torch.randn(G, W, V, generator=g) * std).to(dt).cuda(), (-torch.rand(G, W, generator=g) * 5 - 10).cuda())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,W,V,K", [(1, 1, 1, 1), (1, 1, 5, 3), (2, 3, 7, 4), (1, 4, 1000, 4), (3, 2, 2047, 5), (2, 2, 2049, 8),
                                     (1, 4, 32000, 4), (5, 8, 50257, 16), (1, 64, 333, 64), (2, 5, 100003, 10), (40, 3, 4097, 6),
                                     (1, 1, 60000, 64)])
def test_select(dt, G, W, V, K):
    device()
    check(*data(G, W, V, dt, seed=K), K)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_ties_go_to_the_lowest_index(dt):
    device()
    x = torch.zeros(2, 3, 9001, dtype=dt, device="cuda")          # everything ties
    check(x, torch.full((2, 3), -1.0, device="cuda"), 9)
    x[0, 1, 77] = 3.0
    x[0, 2, 77] = 3.0
    x[0, 2, 8000] = 3.0
    check(x, torch.full((2, 3), -1.0, device="cuda"), 9)
    y, s = data(2, 1, 5000, dt)
    y, s = y.expand(2, 4, 5000).contiguous(), s.expand(2, 4).contiguous()   # four equal beams
    check(y, s, 12)
    check(torch.zeros(2, 64, 500, dtype=dt, device="cuda"), torch.full((2, 64), -1.0, device="cuda"), 64)
    z = torch.tensor([[[0.0, -0.0, 1.0, -0.0]]], dtype=dt, device="cuda")   # both zeros are one value
    assert check(z, torch.zeros(1, 1, device="cuda"), 4)["tokens"].tolist() == [[2, 0, 1, 3]]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 47, 4111])
def test_few_distinct_values(dt, V):
    """Ties across the boundaries of the scan's vectors, whose rows begin at every alignment."""
    device()
    g = torch.Generator().manual_seed(V)
    x = torch.randint(0, 3, (3, 7, V), generator=g).to(dt).cuda()
    x[1, :, : V // 2] = -INF
    x[2, 0] = -1.0
    check(x, -torch.arange(21, dtype=torch.float32, device="cuda").view(3, 7) * 7, 64)
    check(x, -torch.arange(21, dtype=torch.float32, device="cuda").view(3, 7) * 7, 5)


def test_ordered_rows():
    """Ascending logits keep replacing the best so far; descending ones never do."""
    device()
    V = 30011
    up = torch.arange(V, dtype=torch.float32, device="cuda") * 1e-3
    check(torch.stack([up, up.flip(0)])[None].contiguous(), torch.zeros(1, 2, device="cuda"), 64)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_masks_and_dead_beams(dt):
    device()
    low = torch.finfo(dt).min
    x, s = data(8, 4, 3001, dt, seed=3)
    x[0, 0] = -INF                      # a beam with nothing left
    x[1] = -INF                         # a request with nothing left
    x[2, :, 3:] = -INF                  # fewer candidates than asked for
    x[3, 1, 5:] = low                   # masked by the type's lowest value: still candidates, the last ones
    x[3, 0], x[3, 2:], = -INF, -INF
    x[4, 1, 9] = float("nan")
    x[4, 2, 2999] = INF
    s[5, 0], s[5, 1], s[5, 2] = -INF, float("nan"), INF
    s[6] = -INF
    x[7, 2] = low
    check(x, s, 16)
    one = torch.full((1, 2, 4000), -INF, dtype=dt, device="cuda")
    one[0, 1, 3999] = 1.0
    check(one, torch.zeros(1, 2, device="cuda"), 3)


@pytest.mark.parametrize("kind", [torch.bool, torch.uint8])
def test_finished_beams(kind):
    device()
    x, s = data(4, 3, 500, torch.float32, seed=8)
    fin = torch.zeros(4, 3, dtype=torch.bool, device="cuda")
    fin[0, 1] = fin[1] = fin[2, 0] = True
    x[2, 0] = float("nan")              # a finished beam's logits are not looked at
    s[0, 1] = -0.5
    check(x, s, 6, (fin * 3).to(kind) if kind == torch.uint8 else fin, end_token=499)


def test_close_scores_are_told_apart():
    """Beams whose best scores differ by less than fp32 sums of exponentials can tell."""
    device()
    g = torch.Generator().manual_seed(1)
    row = torch.randn(20000, generator=g)
    x = torch.stack([row, row, row[torch.randperm(20000, generator=g)], row])[None].repeat(6, 1, 1).contiguous().cuda()
    s = torch.tensor([-10.0, -10.000001, -10.0, -9.9999990]).repeat(6, 1).cuda()
    x[3, 1, 17] += 1e-4
    x[4, 0] = x[4, 0].flip(0)
    # equal sums in another order may differ in the last bits of fp64: compare the order only where it is defined
    r = ia.beam_select(x, s, 8)
    want, _, _ = P.beam_select(x, s, 8)
    assert ((r["scores"].cpu().double() - want).abs() <= 2e-6 + P.U * want.abs()).all()
    # the lse computed in fp64 on the host decides every order with a gap above 1e-9
    X, S = x.double().cpu(), s.double().cpu()
    lse = torch.logsumexp(X, -1)
    for gi in range(6):
        sc = [float(S[gi, p] + X[gi, p, t] - lse[gi, p]) for p, t in zip(r["parents"][gi].tolist(), r["tokens"][gi].tolist())]
        assert all(a >= b - 1e-9 for a, b in zip(sc, sc[1:]))
        assert abs(sc[-1] - float(want[gi, -1])) < 1e-9


def test_large_scores():
    device()
    x, s = data(2, 4, 4000, torch.float32, seed=2)
    check(x + 5e4, s - 1e5, 8)


def test_select_graph_and_stream():
    device()
    x, s = data(3, 4, 7001, torch.bfloat16)
    a = ia.beam_select(x, s, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = ia.beam_select(x, s, 8, stream=side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c = ia.beam_select(x, s, 8)
    x2, s2 = data(3, 4, 7001, torch.bfloat16, seed=5)
    x.copy_(x2)
    s.copy_(s2)
    graph.replay()
    d = ia.beam_select(x2, s2, 8)
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]) and torch.equal(c[n], d[n])


def plain_reorder(state, parents, sizes, B, G):
    """Section by section: row g*win + parent to row g*wout + j."""
    win, wout = B // G, parents.shape[1]
    out = []
    for part in state.split([n * B for n in sizes]):
        rows = part.view(G, win, -1)
        new = torch.zeros(G, wout, rows.shape[2], device=state.device)
        for g in range(G):
            for j in range(wout):
                p = int(parents[g, j])
                if 0 <= p < win:
                    new[g, j] = rows[g, p]
        out.append(new.flatten())
    return torch.cat(out)


@pytest.mark.parametrize("H,M,dx,dv", [(2, 64, 64, 64), (1, 16, 16, 16), (3, 5, 7, 3), (1, 1, 1, 1), (2, 64, 128, 64)])
@pytest.mark.parametrize("G,win,wout", [(1, 1, 1), (3, 4, 4), (2, 1, 5), (2, 5, 2), (1, 64, 64), (4, 3, 3)])
def test_state_reorder(H, M, dx, dv, G, win, wout):
    device()
    B = G * win
    sizes = [2 * H * M * dx, 2 * H * M * dv, 2 * H * M]
    st = torch.randn(sum(sizes) * B, device="cuda")
    par = torch.randint(-1, win + 1, (G, wout), dtype=torch.int32, device="cuda")
    want = plain_reorder(st, par, sizes, B, G)
    keep = st.clone()
    got = ia.state_reorder(st, par, B, H, M, dx, dv)
    assert torch.equal(got, want) and torch.equal(st, keep)
    if win == wout:
        assert torch.equal(ia.state_reorder(st, par, B, H, M, dx, dv, out=st), want)
        same = torch.arange(win, dtype=torch.int32, device="cuda").repeat(G, 1)
        assert torch.equal(ia.state_reorder(st, same, B, H, M, dx, dv, out=st), want)


@pytest.mark.parametrize("dk,dv", [(64, 64), (5, 3), (128, 64)])
def test_linear_state_reorder(dk, dv):
    device()
    G, W, H = 3, 4, 2
    st = torch.randn(G * W * H * dk * dv, device="cuda")
    par = torch.randint(-1, W, (G, W), dtype=torch.int32, device="cuda")
    want = plain_reorder(st, par, [H * dk * dv], G * W, G)
    assert torch.equal(ia.linear_state_reorder(st, par, G * W, H, dk, dv), want)
    assert torch.equal(ia.linear_state_reorder(st, par, G * W, H, dk, dv, out=st), want)


def test_beam_search_end_to_end():
    """A prompt, its state spread over the beams, then selection and steps through the parents: the best sequence's
    score equals that of scoring its tokens one after the other."""
    device()
    torch.manual_seed(0)
    H, d, V, W, steps = 2, 64, 501, 4, 6
    emb = torch.randn(V, H, 3, d, device="cuda").bfloat16()
    head = (torch.randn(H * d, V, device="cuda") * 0.05)
    g = torch.tensor([-0.05, -0.3], device="cuda")
    norm_w = torch.ones(H * d, device="cuda")

    def logits(o):   # [B,H,d] -> [B,V]
        y = ia.layer_norm_fwd(o.flatten(1).float(), norm_w)["y"]
        return y @ head

    prompt = torch.randint(0, V, (40,), device="cuda")
    e = emb[prompt]                                                     # [N,H,3,d]
    q, k, v = (e[:, :, i].transpose(0, 1)[None].contiguous() for i in range(3))
    pre = ia.linear_prefill_fwd(q, k, v, g, want_state=True)
    state = ia.linear_state_reorder(pre["state"], torch.zeros(1, W, dtype=torch.int32, device="cuda"), 1, H, d, d)
    other = torch.empty_like(state)
    lg = logits(pre["o"][:, :, -1])[:, None].expand(1, W, V).contiguous()
    scores = torch.tensor([[0.0] + [-INF] * (W - 1)], device="cuda")
    history = torch.zeros(1, W, 0, dtype=torch.int64, device="cuda")
    for _ in range(steps):
        r = ia.beam_select(lg, scores, W)
        scores = r["scores"]
        par = r["parents"]
        history = torch.cat([torch.gather(history, 1, par.long()[..., None].expand(1, W, history.shape[2])),
                             r["tokens"].long()[..., None]], 2)
        e = emb[r["tokens"].long().flatten()]
        q, k, v = (e[:, :, i].contiguous() for i in range(3))
        o = ia.linear_decode_step(q, k, v, g, state, parents=par, state_out=other)["o"]
        state, other = other, state
        lg = logits(o)[None].contiguous()
    ia.check_device_errors()
    # score the best history alone
    st = pre["state"].clone()
    row = logits(pre["o"][:, :, -1])
    total = 0.0
    for t in history[0, 0].tolist():
        total += float(torch.log_softmax(row.double(), -1)[0, t])
        e = emb[torch.tensor([t], device="cuda")]
        o = ia.linear_decode_step(*(e[:, :, i].contiguous() for i in range(3)), g, st)["o"]
        row = logits(o)
    # the two runs differ by fp32 matrix products of another batch size: 128 terms of about 0.05
    assert abs(total - float(scores[0, 0])) < steps * 1e-4
    assert torch.isfinite(scores).all() and (scores[0, :-1] >= scores[0, 1:]).all()


def test_two_selections_at_once_and_a_given_workspace():
    device()
    sets = [data(3, 8, 50257, torch.bfloat16, seed=1), data(2, 64, 3001, torch.float32, seed=2)]
    ks = [16, 64]
    want = [ia.beam_select(x, s, k) for (x, s), k in zip(sets, ks)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    works = [torch.full((ia.beam_select_workspace_bytes(*x.shape, k, x.dtype),), 255, dtype=torch.uint8, device="cuda")
             for (x, _), k in zip(sets, ks)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [ia.beam_select(x, s, k, workspace=w, stream=st) for (x, s), k, w, st in zip(sets, ks, works, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(a[n], b[n]) for n in a)
    ia.check_device_errors()
