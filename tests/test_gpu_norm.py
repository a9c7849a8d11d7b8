"""Layer norm on the GPU against its fp64 form."""
import pytest
import torch

import ops_plain as P
import ssm_token_mixer_b200 as ia
from gpu_common import device

pytestmark = pytest.mark.gpu

SIZES = [(1, 1), (1, 2), (3, 31), (5, 32), (2, 33), (1000, 64), (777, 128), (9, 256), (64, 257), (33, 512), (10, 520),
         (17, 777), (130, 1024), (7, 2048), (300, 4096), (3, 4100), (5, 8192), (4, 8200), (3, 9001), (2, 12279), (9, 12280), (2, 12288), (3, 12289),
         (2, 20000), (5000, 96), (700, 1017), (40, 1018), (33, 250), (20, 506), (3, 8185), (5, 8191)]


def data(rows, D, dt, seed=0, mean=0.5):
    g = torch.Generator().manual_seed(seed + rows + D)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return ((rn(rows, D) * 1.5 + mean).to(dt).cuda(), (rn(D) * 0.3 + 1).cuda(), (rn(D) * 0.2).cuda(), rn(rows, D).to(dt).cuda())


def half(dt):
    return torch.finfo(dt).eps / 2


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("params", [True, False])
def test_layer_norm(rows, D, dt, params):
    device()
    x, w, b, dy = data(rows, D, dt)
    if not params:
        w = b = None
    eps = 1e-5
    r = ia.layer_norm_fwd(x, w, b, eps)
    y, mean, rstd, hat = P.layer_norm(x, w, b, eps)
    # Sums of D terms in registers, a warp tree and a few warps: at most E + 5 + 16 roundings per term on the way,
    # E = 24 held values (ceil(D / 512) when rows are read again).
    n = (24 + 5 + 16 if D <= 12280 else D // 512 + 1 + 5 + 16) + 8
    u = n * P.U
    emean = u * x.double().abs().mean(-1)
    assert ((r["mean"].double() - mean).abs() <= emean + 1e-30).all()
    # the variance's terms shift with the mean's error: d var = emean^2 (the linear term sums to zero up to u)
    rel = u + (emean * rstd) ** 2 + 2 * u * emean * rstd
    assert ((r["rstd"].double() - rstd).abs() <= (rel + 4 * P.U) * rstd).all()
    wm = 1.0 if w is None else w.double().abs()
    bm = 0.0 if b is None else b.double().abs()
    ehat = (emean * rstd + 0.0)[:, None] + (rel + 8 * P.U)[:, None] * hat.abs() + P.U * (x.double().abs() * rstd[:, None])
    ey = ehat * wm + 3 * P.U * (hat.abs() * wm + bm)
    ey = ey + half(dt) * (y.abs() + ey) + 1e-30
    assert r["y"].dtype == dt and ((r["y"].double() - y).abs() <= ey).all()

    g = ia.layer_norm_bwd(dy, x, r["mean"], r["rstd"], w)
    dx, dw, db = P.layer_norm_grads(dy, x, w, eps)
    gm = dy.double().abs() * wm
    e1 = u * gm.mean(-1, keepdim=True)
    e2 = (u * (gm * hat.abs()).mean(-1, keepdim=True) + (gm * ehat).mean(-1, keepdim=True))
    c2 = (dy.double() * (1.0 if w is None else w.double()) * hat).mean(-1, keepdim=True).abs()
    edx = rstd[:, None] * (e1 + hat.abs() * e2 + ehat * c2 + 6 * P.U * (gm + gm.mean(-1, keepdim=True) + hat.abs() * c2))
    edx = edx + (rel + 4 * P.U)[:, None] * dx.abs()
    edx = edx + half(dt) * (dx.abs() + edx) + 1e-30
    assert g["dx"].dtype == dt and ((g["dx"].double() - dx).abs() <= edx).all()
    # column sums: rows / blocks per thread, the block's groups, the partial rows by eight lanes
    nr = rows + 20
    edw = (min(nr, 600 + rows // 148) * P.U * (dy.double().abs() * hat.abs()) + dy.double().abs() * ehat).sum(0)
    assert ((g["dweight"].double() - dw).abs() <= edw + 1e-30).all()
    edb = min(nr, 600 + rows // 148) * P.U * dy.double().abs().sum(0)
    assert ((g["dbias"].double() - db).abs() <= edb + 1e-30).all()


def test_gradients_against_differences():
    device()
    x, w, b, dy = data(4, 96, torch.float32)
    r = ia.layer_norm_fwd(x, w, b)
    g = ia.layer_norm_bwd(dy, x, r["mean"], r["rstd"], w)
    gen = torch.Generator().manual_seed(3)
    e = 1e-5

    def loss(x, w, b):
        return (P.layer_norm(x, w, b, 1e-5)[0] * dy.double()).sum()

    base = {"x": x.double(), "w": w.double(), "b": b.double()}
    for name, key in (("x", "dx"), ("w", "dweight"), ("b", "dbias")):
        d = torch.randn(base[name].shape, generator=gen).cuda().double()
        want = (loss(**{**base, name: base[name] + e * d}) - loss(**{**base, name: base[name] - e * d})) / (2 * e)
        mag = (g[key].double().abs() * d.abs()).sum()
        assert (want - (g[key].double() * d).sum()).abs() <= 1e-5 * mag


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 777, 2048, 13000])
def test_in_place_and_large_offset(dt, D):
    device()
    x, w, b, dy = data(37, D, dt, mean=100.0)   # the variance of values far from zero
    want = ia.layer_norm_fwd(x, w, b)
    y, _, _, _ = P.layer_norm(x, w, b, 1e-5)
    assert ((want["y"].double() - y).norm() / y.norm()) < (3e-4 if dt == torch.float32 else 4e-3)
    grad = ia.layer_norm_bwd(dy, x, want["mean"], want["rstd"], w)
    for target in ("dy", "x"):
        c = {"dy": dy.clone(), "x": x.clone()}
        again = ia.layer_norm_bwd(c["dy"], c["x"], want["mean"], want["rstd"], w, dx=c[target])
        for n in grad:
            assert torch.equal(again[n], grad[n])
    z = x.clone()
    assert torch.equal(ia.layer_norm_fwd(z, w, b, y=z)["y"], want["y"])
    none = ia.layer_norm_bwd(dy, x, want["mean"], want["rstd"], w, want_params=False)
    assert none["dweight"] is None and torch.equal(none["dx"], grad["dx"])


def test_rows_do_not_mix_and_shapes():
    device()
    x, w, b, dy = data(60, 128, torch.bfloat16)
    clean = ia.layer_norm_fwd(x, w, b)["y"]
    x[7, 5] = float("nan")
    x[9, 0] = float("inf")
    r = ia.layer_norm_fwd(x.view(3, 4, 5, 128), w, b)
    assert r["mean"].shape == (3, 4, 5)
    y = r["y"].view(60, 128)
    keep = [i for i in range(60) if i not in (7, 9)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[7].float()).all() and torch.isnan(y[9].float()).any()


def test_constant_rows_and_graph():
    device()
    x = torch.full((5, 300), 2.5, device="cuda")
    r = ia.layer_norm_fwd(x)
    assert torch.equal(r["y"], torch.zeros_like(x))
    dy = torch.randn(5, 300, device="cuda")
    w = torch.ones(300, device="cuda")
    graph = torch.cuda.CUDAGraph()
    want = ia.layer_norm_bwd(dy, x, r["mean"], r["rstd"], w)
    with torch.cuda.graph(graph):
        got = ia.layer_norm_bwd(dy, x, r["mean"], r["rstd"], w)
    graph.replay()
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(want[n], got[n])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_backward_captured_and_two_calls_at_once(dt):
    device()
    sets = [data(700, 320, dt), data(333, 777, dt)]
    stats = [ia.layer_norm_fwd(x, w, b) for x, w, b, _ in sets]
    run = lambda i, **kw: ia.layer_norm_bwd(sets[i][3], sets[i][0], stats[i]["mean"], stats[i]["rstd"], sets[i][1], **kw)  # noqa: E731
    want = [run(0), run(1)]
    graph = torch.cuda.CUDAGraph()
    work = torch.empty(ia.layer_norm_bwd_workspace_bytes(700, 320, dt), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = run(0, workspace=work)
    for t in got.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[n], want[0][n]) for n in got)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        both = [run(i, stream=st) for i, st in enumerate(streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(both[i][n], want[i][n]) for i in (0, 1) for n in want[i])
