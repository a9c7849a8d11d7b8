"""Linear attention with one decay per head on the GPU, against the fp64 recurrence."""
import pytest
import torch

import ops_plain as P
import ssm_token_mixer_b200 as ia
from gpu_common import device

pytestmark = pytest.mark.gpu


def make(B, H, N, dk, dv, dt, seed=0, decay=None, state=False, grad=False, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = {"q": rn(B, H, N, dk).to(dt), "k": rn(B, H, N, dk).to(dt), "v": rn(B, H, N, dv).to(dt)}
    if decay is None:
        t["g"] = torch.log1p(-torch.exp2(-(1.5 + 10.0 * torch.rand(H, generator=g))))
    else:
        t["g"] = torch.full((H,), float(decay))
    t["s"] = rn(B, H, dk, dv) * 3 if state else None
    if grad:
        t["dO"] = rn(B, H, N, dv).to(dt)
    return {k: None if v is None else v.to(dev) for k, v in t.items()}


def within(got, want, bound):
    over = (got.double() - want).abs() - bound
    assert torch.isfinite(got.double()).all()
    assert (over <= 0).all(), f"off by up to {over.max().item():.3g} over the bound"


def is_tc(shape, dt):
    return ia.linear_path(*shape, dt) == "tensor_core"


SHAPES = [  # B, H, N, d_k, d_v
    (1, 1, 1, 64, 64), (2, 3, 5, 64, 64), (1, 2, 63, 64, 64), (1, 2, 64, 64, 64), (2, 1, 127, 64, 64),
    (1, 3, 128, 64, 64), (1, 1, 129, 64, 64), (2, 2, 257, 64, 64), (1, 1, 1000, 64, 64), (1, 2, 300, 128, 128),
    (2, 1, 200, 64, 128), (1, 2, 200, 128, 64), (1, 1, 2049, 128, 128), (3, 50, 130, 64, 64),
    (1, 2, 70, 16, 16), (1, 1, 33, 1, 1), (2, 1, 100, 7, 13), (1, 1, 90, 96, 65), (1, 2, 150, 256, 200), (1, 1, 40, 129, 256),
]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("with_state", [False, True])
def test_prefill(shape, dt, with_state):
    device()
    B, H, N, dk, dv = shape
    t = make(*shape, dt, seed=N, state=with_state)
    r = ia.linear_prefill_fwd(t["q"], t["k"], t["v"], t["g"], state_in=t["s"], want_state=True)
    ia.check_device_errors()
    o, bo, S, bS = P.linear_bounds(t["q"], t["k"], t["v"], t["g"], dk ** -0.5, is_tc(shape, dt), t["s"])
    assert r["o"].dtype == dt and r["o"].shape == (B, H, N, dv)
    within(r["o"], o, bo)
    within(r["state"].view_as(S), S, bS)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_fwd_bwd(shape, dt):
    device()
    t = make(*shape, dt, seed=N_of(shape) + 7, grad=True)
    sc = 0.3
    r = ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"], scale=sc)
    ia.check_device_errors()
    q, k, v, dO, g, tc = t["q"], t["k"], t["v"], t["dO"], t["g"], is_tc(shape, dt)
    for name, (x, y, z, rev) in {"o": (q, k, v, False), "dq": (dO, v, k, False), "dk": (v, dO, q, True),
                                 "dv": (k, q, dO, True)}.items():
        want, bound, _, _ = P.linear_bounds(x, y, z, g, sc, tc, reverse=rev)
        assert r[name].dtype == dt
        within(r[name], want, bound)


def N_of(shape):
    return shape[2]


def test_gradients_against_differences():
    """The analytic gradients of sum(o * dO) against central differences of the fp64 recurrence."""
    device()
    t = make(1, 2, 40, 64, 64, torch.float32, seed=3, grad=True)
    r = ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"], scale=1.0)

    def loss(q, k, v):
        return (P.recurrence(q, k, v, t["g"])[0] * t["dO"].double()).sum()

    gen = torch.Generator().manual_seed(1)
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        d = torch.randn(t[name].shape, generator=gen).to(t[name].device).double()
        e = 1e-4
        args = {n: t[n].double() for n in "qkv"}
        up = loss(**{**args, name: args[name] + e * d})
        dn = loss(**{**args, name: args[name] - e * d})
        want = ((up - dn) / (2 * e)).item()   # o is bilinear in any one input: no truncation error
        got = (r[key].double() * d).sum().item()
        mag = (r[key].double().abs() * d.abs()).sum().item()
        assert abs(got - want) <= 1e-5 * mag


@pytest.mark.parametrize("decay", [0.0, -1e-6, -0.01, -3.0, -80.0, -1e4, float("-inf")])
@pytest.mark.parametrize("dt,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 24)])
def test_decays(decay, dt, d):
    device()
    shape = (1, 2, 333, d, d)
    t = make(*shape, dt, seed=11, decay=decay, grad=True, state=True)
    tc = is_tc(shape, dt)
    r = ia.linear_prefill_fwd(t["q"], t["k"], t["v"], t["g"], state_in=t["s"], want_state=True)
    b = ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"])
    ia.check_device_errors()
    o, bo, S, bS = P.linear_bounds(t["q"], t["k"], t["v"], t["g"], d ** -0.5, tc, t["s"])
    within(r["o"], o, bo)
    within(r["state"].view_as(S), S, bS)
    dk, bdk, _, _ = P.linear_bounds(t["v"], t["dO"], t["q"], t["g"], d ** -0.5, tc, reverse=True)
    within(b["dk"], dk, bdk)


@pytest.mark.parametrize("bad", [1e-3, float("nan"), float("inf")])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_positive_or_nan_decay_is_reported(bad, dt):
    device()
    t = make(1, 2, 20, 64, 64, dt)
    t["g"][1] = bad
    ia.linear_prefill_fwd(t["q"], t["k"], t["v"], t["g"])
    with pytest.raises(ia.IAError) as e:
        ia.check_device_errors()
    assert e.value.status == 6
    ia.check_device_errors()   # cleared
    st = torch.zeros(2 * 64 * 64, device="cuda")
    ia.linear_decode_step(t["q"][:, :, 0].contiguous(), t["k"][:, :, 0].contiguous(), t["v"][:, :, 0].contiguous(),
                          t["g"], st)
    with pytest.raises(ia.IAError):
        ia.check_device_errors()


@pytest.mark.parametrize("dt,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 40)])
@pytest.mark.parametrize("which", ["q", "k", "v", "dO"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_token_reaches_nothing_before_it(dt, d, which, value):
    device()
    N, u = 300, 171
    t = make(1, 2, N, d, d, dt, seed=5, grad=True)
    clean = ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"])
    t[which][0, 1, u, d // 2] = value
    r = ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"])
    ia.check_device_errors()
    for name in ("o", "dq"):   # forward in time
        assert torch.equal(r[name][0, 0], clean[name][0, 0])
        assert torch.equal(r[name][0, 1, :u], clean[name][0, 1, :u])
    for name in ("dk", "dv"):
        assert torch.equal(r[name][0, 0], clean[name][0, 0])
        assert torch.equal(r[name][0, 1, u + 1:], clean[name][0, 1, u + 1:])
    if which == "v":
        assert not torch.isfinite(r["o"][0, 1, u:, d // 2].float()).any()


@pytest.mark.parametrize("dt,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 33)])
def test_prefill_in_two_calls_then_decode(dt, d):
    """A prompt in two pieces, then token by token, against the whole sequence in fp64."""
    device()
    B, H, N, n1, n2 = 2, 2, 290, 131, 270
    t = make(B, H, N, d, d, dt, seed=9)
    piece = lambda a, b: [t[n][:, :, a:b].contiguous() for n in "qkv"]  # noqa: E731
    r1 = ia.linear_prefill_fwd(*piece(0, n1), t["g"], want_state=True)
    r2 = ia.linear_prefill_fwd(*piece(n1, n2), t["g"], state_in=r1["state"], want_state=True)
    outs, st = [r1["o"], r2["o"]], r2["state"]
    for i in range(n2, N):
        q, k, v = (t[n][:, :, i].contiguous() for n in "qkv")
        outs.append(ia.linear_decode_step(q, k, v, t["g"], st)["o"][:, :, None])
    ia.check_device_errors()
    o, bo, S, bS = P.linear_bounds(t["q"], t["k"], t["v"], t["g"], d ** -0.5, is_tc((B, H, n1, d, d), dt))
    within(torch.cat(outs, 2), o, bo)
    within(st.view_as(S), S, bS)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 1, 1), (1, 16, 128, 128), (3, 5, 64, 128), (2, 3, 7, 9), (64, 4, 128, 64),
                                       (2, 2, 256, 256), (1, 3, 200, 100), (160, 1, 33, 132)])
@pytest.mark.parametrize("apart", [False, True])
def test_decode(dt, B, H, dk, dv, apart):
    device()
    t = make(B, H, 1, dk, dv, dt, seed=dk, state=True)
    q, k, v = (t[n][:, :, 0].contiguous() for n in "qkv")
    st = t["s"].clone()
    out = torch.full_like(st, 7.0) if apart else None
    r = ia.linear_decode_step(q, k, v, t["g"], st, scale=0.7, state_out=out)
    ia.check_device_errors()
    o, bo, S, bS = P.linear_bounds(t["q"], t["k"], t["v"], t["g"], 0.7, False, t["s"])
    within(r["o"][:, :, None], o, bo)
    within(r["state"].view_as(S), S, bS)
    assert torch.equal(st, t["s"]) if apart else r["state"] is st


@pytest.mark.parametrize("W", [1, 2, 5])
def test_decode_through_parents(W):
    device()
    G, H, d = 3, 2, 64
    B = G * W
    t = make(B, H, 1, d, d, torch.bfloat16, seed=2, state=True)
    q, k, v = (t[n][:, :, 0].contiguous() for n in "qkv")
    par = torch.randint(0, W, (G, W), dtype=torch.int32, device="cuda")
    par[1, W - 1] = -1
    par[2, 0] = W
    out = torch.empty(t["s"].numel(), device="cuda")
    r = ia.linear_decode_step(q, k, v, t["g"], t["s"], parents=par, state_out=out)
    ia.check_device_errors()
    ok = (par >= 0) & (par < W)
    rows = (torch.arange(G, device="cuda")[:, None] * W + par.clamp(0, W - 1)).flatten().long()
    src = torch.where(ok.flatten()[:, None, None, None], t["s"][rows], torch.zeros((), device="cuda"))
    alone = ia.linear_decode_step(q, k, v, t["g"], src.flatten().clone())   # in place on a copy
    assert torch.equal(r["o"], alone["o"]) and torch.equal(r["state"], alone["state"])
    # the same through a reordering pass
    moved = ia.linear_state_reorder(t["s"].flatten(), par, B, H, d, d)
    assert torch.equal(moved, src.flatten())


def test_equal_calls_give_equal_bits_and_streams_and_graphs():
    device()
    t = make(2, 3, 700, 64, 64, torch.bfloat16, seed=4, grad=True)
    a = ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"], stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"])
    for x in c.values():
        x.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n])
    ia.check_device_errors()


@pytest.mark.parametrize("dt,d,N", [(torch.bfloat16, 128, 5000), (torch.bfloat16, 64, 3001), (torch.float32, 48, 2000)])
def test_few_long_sequences_run_in_segments(dt, d, N):
    device()
    shape = (1, 2, N, d, d)
    assert ia.linear_prefill_segments(*shape, dt) > 2 and ia.linear_fwd_bwd_segments(*shape, dt) > 2
    t = make(*shape, dt, seed=6, state=True, grad=True)
    t["g"][0] = -1e-4
    ws = torch.full((max(1, ia.linear_prefill_workspace_bytes(*shape, dt)),), 255, dtype=torch.uint8, device="cuda")
    r = ia.linear_prefill_fwd(t["q"], t["k"], t["v"], t["g"], state_in=t["s"], want_state=True, workspace=ws)
    b = ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"])
    ia.check_device_errors()
    tc = is_tc(shape, dt)
    o, bo, S, bS = P.linear_bounds(t["q"], t["k"], t["v"], t["g"], d ** -0.5, tc, t["s"])
    within(r["o"], o, bo)
    within(r["state"].view_as(S), S, bS)
    q, k, v, dO, g = t["q"], t["k"], t["v"], t["dO"], t["g"]
    for name, (x, y, z, rev) in {"o": (q, k, v, False), "dq": (dO, v, k, False), "dk": (v, dO, q, True),
                                 "dv": (k, q, dO, True)}.items():
        want, bound, _, _ = P.linear_bounds(x, y, z, g, d ** -0.5, tc, reverse=rev)
        within(b[name], want, bound)


@pytest.mark.parametrize("shape", [(1, 2, 1000, 64, 64), (1, 1, 1300, 128, 128), (2, 1, 900, 64, 128), (1, 2, 650, 128, 64)])
@pytest.mark.parametrize("segments", [1, 2, 3, 5])
def test_every_segment_count_and_with_or_without_the_state(shape, segments, monkeypatch):
    """The tensor-core passes in their forms: whole and in segments, the final state taken or not, widths alike or not."""
    device()
    monkeypatch.setenv("IA_LINEAR_SEGMENTS", str(segments))
    assert 1 <= ia.linear_prefill_segments(*shape, torch.bfloat16) <= segments
    t = make(*shape, torch.bfloat16, seed=segments, state=True, grad=True)
    q, k, v, dO, g = t["q"], t["k"], t["v"], t["dO"], t["g"]
    scale = shape[3] ** -0.5
    o, bo, S, bS = P.linear_bounds(q, k, v, g, scale, True, t["s"])
    for want in (False, True):
        r = ia.linear_prefill_fwd(q, k, v, g, state_in=t["s"], want_state=want)
        within(r["o"], o, bo)
        if want:
            within(r["state"].view_as(S), S, bS)
    b = ia.linear_fwd_bwd(q, k, v, g, dO)
    ia.check_device_errors()
    for name, (x, y, z, rev) in {"o": (q, k, v, False), "dq": (dO, v, k, False), "dk": (v, dO, q, True),
                                 "dv": (k, q, dO, True)}.items():
        want, bound, _, _ = P.linear_bounds(x, y, z, g, scale, True, reverse=rev)
        within(b[name], want, bound)


@pytest.mark.parametrize("dt,d,N", [(torch.bfloat16, 64, 1500), (torch.bfloat16, 128, 1500), (torch.float32, 40, 400)])
def test_two_calls_at_once(dt, d, N):
    """Calls on two streams, each with memory of its own, give what they give one after the other."""
    device()
    a, b = (make(1, 2, N, d, d, dt, seed=s, grad=True) for s in (1, 2))
    want = [ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"]) for t in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [ia.linear_fwd_bwd(t["q"], t["k"], t["v"], t["g"], t["dO"], stream=st) for t, st in zip((a, b), streams)]
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            for n in x:
                assert torch.equal(x[n], y[n])
    ia.check_device_errors()


def test_one_tensor_in_several_roles():
    device()
    t = make(2, 2, 300, 64, 64, torch.bfloat16, seed=9)
    x, g = t["q"], t["g"]
    r = ia.linear_prefill_fwd(x, x, x, g, want_state=True)
    b = ia.linear_fwd_bwd(x, x, x, g, x)
    c = x.clone()
    r2 = ia.linear_prefill_fwd(x, c, c.clone(), g, want_state=True)
    b2 = ia.linear_fwd_bwd(x, c, c.clone(), g, c.clone())
    for n in r:
        assert torch.equal(r[n], r2[n])
    for n in b:
        assert torch.equal(b[n], b2[n])
    ia.check_device_errors()


def test_decode_captured_through_parents():
    """Steps of a beam search in one graph: two buffers take turns, the parents are what their tensor holds at replay."""
    device()
    B, H, d, W = 6, 2, 64, 3
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(B, H, d, generator=g).bfloat16().cuda() for _ in range(3))
    decay = torch.tensor([-0.1, -0.5]).cuda()
    start = torch.randn(B * H * d * d, generator=g).cuda()
    bufs = [start.clone(), torch.empty_like(start)]
    parents = torch.zeros(B // W, W, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a = ia.linear_decode_step(q, k, v, decay, bufs[0], state_out=bufs[1], parents=parents)
        b = ia.linear_decode_step(k, q, v, decay, bufs[1], state_out=bufs[0], parents=parents)
    for seed in range(3):
        parents.copy_(torch.randint(0, W, (B // W, W), generator=torch.Generator().manual_seed(seed), dtype=torch.int32))
        now = bufs[0].clone()
        graph.replay()
        torch.cuda.synchronize()
        other = torch.empty_like(now)
        x = ia.linear_decode_step(q, k, v, decay, now, state_out=other, parents=parents)
        y = ia.linear_decode_step(k, q, v, decay, other, state_out=now, parents=parents)
        assert torch.equal(a["o"], x["o"]) and torch.equal(b["o"], y["o"]) and torch.equal(bufs[0], now)
    ia.check_device_errors()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_training_step_through_norm_and_attention(dt):
    """Layer norm, linear attention and both backward passes as one step, against autograd of the definitions in fp64."""
    device()
    B, N, H, d = 2, 150, 3, 64
    D = H * d
    gen = torch.Generator().manual_seed(12)
    x = torch.randn(B, N, D, generator=gen).to(dt).cuda()
    w, b = (torch.randn(D, generator=gen) * 0.2 + 1).cuda(), (torch.randn(D, generator=gen) * 0.1).cuda()
    dO = torch.randn(B, H, N, d, generator=gen).to(dt).cuda()
    decay = torch.tensor([-0.02, -0.3, 0.0]).cuda()

    n = ia.layer_norm_fwd(x, w, b)
    h = n["y"].view(B, N, H, d).transpose(1, 2).contiguous()
    r = ia.linear_fwd_bwd(h, h, h, decay, dO)
    dh = r["dq"].float() + r["dk"].float() + r["dv"].float()
    dy = dh.transpose(1, 2).reshape(B, N, D).to(dt)
    g = ia.layer_norm_bwd(dy, x, n["mean"], n["rstd"], w)
    ia.check_device_errors()

    x64, w64, b64 = (t.double().requires_grad_() for t in (x, w, b))
    y = torch.nn.functional.layer_norm(x64, (D,), w64, b64)
    q = y.view(B, N, H, d).transpose(1, 2)
    t = torch.arange(N, device="cuda")
    far = (t[:, None] - t[None]).double()
    mask = torch.where(far >= 0, torch.exp(decay.double()[:, None, None] * far.clamp(min=0)), 0.0)
    o = d ** -0.5 * ((q @ q.transpose(-1, -2)) * mask) @ q
    (o * dO.double()).sum().backward()
    # fp32: a path sums at most 450 terms (150 tokens, 64 and 192 columns, and what is around them), 450 U of a sum of
    # magnitudes some 20 times the sum of random signs: 5.4e-4.  bf16: h, P, o, the three gradients, dy and dx are
    # rounded, eight times half a unit 2^-9 of the magnitudes a value is formed from, up to three in a row on a path
    # whose magnitudes are a few times its value; as norms, 8 * 2^-9 * 3.
    tol = 5.4e-4 if dt == torch.float32 else 8 * 2.0 ** -9 * 3
    for name, got, want in (("o", r["o"], o), ("dx", g["dx"], x64.grad), ("dweight", g["dweight"], w64.grad),
                            ("dbias", g["dbias"], b64.grad)):
        assert (got.double() - want).norm() <= tol * want.norm(), name
