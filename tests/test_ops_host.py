"""Argument checks of linear attention, layer norm and beam search, on the CPU: the C-ABI refuses bad arguments before
any launch, and the binding checks every tensor before the library sees its address."""
import ctypes

import pytest
import torch

import ssm_token_mixer_b200 as ia

P = 0x10000            # aligned, never dereferenced: validation fails first, or the injected failure stops the call
ODD = 0x10008
BAD_ARG, UNSUPPORTED, WORKSPACE, CUDA = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from ssm_token_mixer_b200 import build
    build.build()
    return ia.load_library()


@pytest.fixture
def no_launch(monkeypatch):
    monkeypatch.setenv("IA_INJECT_LAUNCH_FAILURE", "1")   # valid calls return IA_ERR_CUDA and launch nothing


def lshape(B=2, H=3, N=100, dk=64, dv=64, dt=1):
    return ia.IALinearShape(B, H, N, dk, dv, dt)


def linear_prefill(lib, s, q=P, g=P, scale=0.1, sin=None, o=P, sout=None, ws=P, wsb=1 << 40):
    return lib.ia_linear_prefill_fwd(ctypes.byref(s), q, P, P, g, scale, sin, o, sout, ws, wsb, None)


def linear_train(lib, s, dO=P, dq=P, scale=0.1, ws=P, wsb=1 << 40):
    return lib.ia_linear_fwd_bwd(ctypes.byref(s), P, P, P, P, scale, dO, P, dq, P, P, ws, wsb, None)


def linear_decode(lib, s, sin=P, parents=None, beams=0, sout=P, o=P, scale=0.1):
    return lib.ia_linear_decode_step(ctypes.byref(s), P, P, P, P, scale, sin, parents, beams, sout, o, None)


def test_linear_refusals(lib, no_launch):
    assert linear_prefill(lib, lshape()) == CUDA
    assert linear_train(lib, lshape()) == CUDA
    assert linear_decode(lib, lshape()) == CUDA
    for bad in (dict(B=0), dict(H=-1), dict(N=0), dict(dk=0), dict(dv=-3), dict(dt=2)):
        assert linear_prefill(lib, lshape(**bad)) == BAD_ARG, bad
        assert linear_train(lib, lshape(**bad)) == BAD_ARG, bad
        if "N" not in bad:
            assert linear_decode(lib, lshape(**bad)) == BAD_ARG, bad
    for bad in (dict(dk=257), dict(dv=300)):
        assert linear_prefill(lib, lshape(**bad)) == UNSUPPORTED
        assert linear_train(lib, lshape(**bad)) == UNSUPPORTED
        assert linear_decode(lib, lshape(**bad)) == UNSUPPORTED
    for kw in (dict(q=None), dict(g=None), dict(o=None), dict(q=ODD), dict(sin=ODD), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(sin=P, sout=P)):
        assert linear_prefill(lib, lshape(), **kw) == BAD_ARG, kw
    sb = lib.ia_linear_state_bytes(ctypes.byref(lshape()))
    assert linear_prefill(lib, lshape(), sin=P, sout=P + sb - 16) == BAD_ARG      # overlapping states
    assert linear_prefill(lib, lshape(), sin=P, sout=P + sb) == CUDA
    for kw in (dict(dO=None), dict(dq=None), dict(dO=ODD), dict(scale=float("nan"))):
        assert linear_train(lib, lshape(), **kw) == BAD_ARG, kw
    assert linear_prefill(lib, lshape(B=1 << 15, H=1 << 15)) == BAD_ARG          # too many streams


def test_linear_decode_parents(lib, no_launch):
    s = lshape(B=6)
    sb = lib.ia_linear_state_bytes(ctypes.byref(s))
    assert sb == 6 * 3 * 64 * 64 * 4
    assert linear_decode(lib, s, sin=P, sout=P + sb, parents=P, beams=3) == CUDA
    assert linear_decode(lib, s, sin=P, sout=P, parents=P, beams=3) == BAD_ARG    # a state may have several followers
    assert linear_decode(lib, s, sin=P, sout=P + 64, parents=P, beams=3) == BAD_ARG
    assert linear_decode(lib, s, sin=P, sout=P + 64) == BAD_ARG                   # neither in place nor apart
    for beams in (0, -1, 4):
        assert linear_decode(lib, s, sin=P, sout=P + sb, parents=P, beams=beams) == BAD_ARG
    assert linear_decode(lib, s, sin=P, sout=P + sb, parents=P + 2, beams=3) == BAD_ARG


def test_linear_workspace_and_plan(lib, no_launch, monkeypatch):
    s = lshape(B=1, H=2, N=5000)
    need = lib.ia_linear_prefill_workspace_bytes(ctypes.byref(s))
    n = lib.ia_linear_prefill_segments(ctypes.byref(s))
    assert n > 1 and need == (n - 1) * lib.ia_linear_state_bytes(ctypes.byref(s))
    assert linear_prefill(lib, s, wsb=need - 1) == WORKSPACE
    assert linear_prefill(lib, s, ws=None) == WORKSPACE
    assert linear_prefill(lib, s, wsb=need) == CUDA
    need = lib.ia_linear_fwd_bwd_workspace_bytes(ctypes.byref(s))
    assert linear_train(lib, s, wsb=need - 1) == WORKSPACE and linear_train(lib, s, wsb=need) == CUDA
    assert ia.linear_prefill_segments(64, 16, 64, 64, 64, "bf16") == 1            # one chunk: nothing to cut
    assert ia.linear_prefill_workspace_bytes(64, 16, 64, 64, 64, "bf16") == 0
    assert ia.linear_path(1, 1, 9, 64, 128, "bf16") == "tensor_core"
    assert ia.linear_path(1, 1, 9, 64, 96, "bf16") == "sequential"
    assert ia.linear_path(1, 1, 9, 64, 64, "f32") == "sequential"
    assert ia.linear_path(1, 1, 9, 0, 64, "f32") is None and ia.linear_path(1, 1, 9, 64, 999, "f32") is None
    for forced in (1, 2, 3, 7, 40, 1000):
        monkeypatch.setenv("IA_LINEAR_SEGMENTS", str(forced))
        got = ia.linear_prefill_segments(1, 1, 5000, 64, 64, "bf16")               # 40 chunks of 128
        assert 1 <= got <= min(forced, 40)
        cps = -(-40 // got)
        assert (got - 1) * cps < 40 <= got * cps                                   # no empty segment


@pytest.mark.parametrize("dt", [0, 1])
def test_norm_refusals(lib, no_launch, dt):
    def fwd(rows=4, D=10, d=dt, x=P, w=P, eps=1e-5, y=P, mean=P):
        return lib.ia_layer_norm_fwd(rows, D, d, x, w, P, eps, y, mean, P, None)

    def bwd(rows=4, D=10, d=dt, dy=P, x=P, mean=P, dx=P, dw=P, ws=P, wsb=1 << 40):
        return lib.ia_layer_norm_bwd(rows, D, d, dy, x, P, mean, P, dx, dw, P, ws, wsb, None)

    assert fwd() == CUDA and bwd() == CUDA and fwd(w=None, mean=None) == CUDA
    for f in (fwd, bwd):
        for kw in (dict(rows=0), dict(rows=-1), dict(D=0), dict(d=5), dict(x=None), dict(x=ODD), dict(rows=1 << 60)):
            assert f(**kw) == BAD_ARG, kw
        assert f(D=(1 << 24) + 1) == UNSUPPORTED
    assert fwd(eps=-1e-9) == BAD_ARG and fwd(eps=float("nan")) == BAD_ARG and fwd(eps=float("inf")) == BAD_ARG
    assert fwd(y=None) == BAD_ARG and bwd(dy=None) == BAD_ARG and bwd(dx=None) == BAD_ARG and bwd(mean=None) == BAD_ARG
    need = lib.ia_layer_norm_bwd_workspace_bytes(4, 10, dt)
    assert need > 0 and bwd(wsb=need - 1) == WORKSPACE and bwd(ws=None) == WORKSPACE and bwd(wsb=need) == CUDA
    assert lib.ia_layer_norm_bwd(4, 10, dt, P, P, P, P, P, P, None, None, None, 0, None) == CUDA   # no sums: no workspace
    assert lib.ia_layer_norm_bwd_workspace_bytes(0, 10, dt) == 0


@pytest.mark.parametrize("dt", [0, 1])
def test_beam_refusals(lib, no_launch, dt):
    def call(G=2, W=3, V=50, K=4, d=dt, x=P, s=P, fin=None, end=0, out=P, ws=P, wsb=1 << 40):
        return lib.ia_beam_select(G, W, V, K, d, x, s, fin, end, out, P, P, ws, wsb, None)

    assert call() == CUDA and call(W=64, K=64) == CUDA and call(V=1, K=64) == CUDA
    for kw in (dict(G=0), dict(W=0), dict(W=65), dict(V=0), dict(K=0), dict(K=65), dict(d=3), dict(x=None), dict(s=None),
               dict(out=None), dict(x=ODD), dict(fin=P, end=50), dict(fin=P, end=-1)):
        assert call(**kw) == BAD_ARG, kw
    assert call(fin=P + 3, end=49) == CUDA and call(end=-7) == CUDA      # bytes need no alignment; no end token without finished
    need = lib.ia_beam_select_workspace_bytes(2, 3, 50, 4, dt)
    assert need > 0 and call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE and call(wsb=need) == CUDA
    assert lib.ia_beam_select_workspace_bytes(2, 3, 50, 0, dt) == 0


def test_reorder_refusals(lib, no_launch):
    s = ia.IAShape(6, 2, 1, 8, 4, 16, 0)
    row = lib.ia_state_bytes(ctypes.byref(s)) // 6

    def call(shape=s, win=3, wout=3, par=P, src=P, dst=P + 6 * row):
        return lib.ia_state_reorder(ctypes.byref(shape), win, wout, par, src, dst, None)

    assert call() == CUDA and call(dst=P) == CUDA and call(wout=5) == CUDA and call(win=1, wout=64) == CUDA
    for kw in (dict(win=0), dict(win=4), dict(win=65), dict(wout=0), dict(wout=65), dict(par=None), dict(src=None),
               dict(dst=None), dict(src=ODD), dict(par=P + 1), dict(dst=P, wout=2), dict(dst=P + row),
               dict(src=P + row, dst=P), dict(shape=ia.IAShape(0, 2, 1, 8, 4, 16, 0))):
        assert call(**kw) == BAD_ARG, kw
    # more beams out than in: the destination is longer than the source
    assert call(win=1, wout=2, src=P + 11 * row, dst=P) == BAD_ARG and call(win=1, wout=2, src=P + 12 * row, dst=P) == CUDA
    ls = lshape(B=6)
    assert lib.ia_linear_state_reorder(ctypes.byref(ls), 3, 3, P, P, P, None) == CUDA
    assert lib.ia_linear_state_reorder(ctypes.byref(ls), 4, 4, P, P, P, None) == BAD_ARG
    assert lib.ia_linear_state_reorder(ctypes.byref(lshape(dk=999)), 1, 1, P, P, P, None) == BAD_ARG


# ------------------------------------------------------------------ the binding
def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def seq(B=2, H=3, N=5, dk=8, dv=4):
    return [bf(B, H, N, dk), bf(B, H, N, dk), bf(B, H, N, dv), torch.zeros(H)]


def test_binding_wants_cuda_tensors(lib):
    q, k, v, g = seq()
    x = torch.zeros(4, 8)
    st = torch.zeros(2 * 3 * 8 * 4)
    par = torch.zeros(1, 2, dtype=torch.int32)
    for call in (lambda: ia.linear_prefill_fwd(q, k, v, g), lambda: ia.linear_fwd_bwd(q, k, v, g, v),
                 lambda: ia.linear_decode_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, st), lambda: ia.layer_norm_fwd(x),
                 lambda: ia.layer_norm_bwd(x, x, x[:, 0].contiguous(), x[:, 0].contiguous()),
                 lambda: ia.beam_select(torch.zeros(1, 2, 9), torch.zeros(1, 2), 2),
                 lambda: ia.linear_state_reorder(st, par, 2, 3, 8, 4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_shapes_and_dtypes(lib):
    q, k, v, g = seq()
    bad = [((q, k[:, :, :4], v, g), ValueError), ((q, k, v[:1], g), ValueError), ((q, k.float(), v, g), TypeError),
           ((q, k, v.float(), g), TypeError), ((q, k, v, g[:2]), ValueError), ((q, k, v, g.double()), TypeError),
           ((q[0], k, v, g), ValueError), ((q.half(), k, v, g), TypeError), ((q, k, None, g), TypeError), ((None, k, v, g), TypeError)]
    for args, err in bad:
        with pytest.raises(err):
            ia.linear_prefill_fwd(*args)
    with pytest.raises(ValueError):
        ia.linear_prefill_fwd(q, k, v, g, state_in=torch.zeros(5))
    with pytest.raises(TypeError):
        ia.linear_prefill_fwd(q, k, v, g, state_in=bf(2, 3, 8, 4))
    with pytest.raises(ValueError):
        ia.linear_fwd_bwd(q, k, v, g, q)
    t = [x[:, :, 0].contiguous() for x in (q, k, v)]
    st = torch.zeros(2 * 3 * 8 * 4)
    with pytest.raises(ValueError, match="state_out"):
        ia.linear_decode_step(*t, g, st, parents=torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        ia.linear_decode_step(*t, g, st, parents=torch.zeros(1, 2), state_out=st.clone())
    with pytest.raises(ValueError):
        ia.linear_decode_step(*t, g, st[1:])
    x = torch.zeros(3, 8)
    for kw, err in ((dict(weight=torch.zeros(7)), ValueError), (dict(bias=bf(8)), TypeError), (dict(y=torch.zeros(3, 7)), ValueError)):
        with pytest.raises(err):
            ia.layer_norm_fwd(x, **kw)
    with pytest.raises(ValueError):
        ia.layer_norm_fwd(torch.zeros(0, 8))
    with pytest.raises(TypeError):
        ia.layer_norm_fwd(x.double())
    m = torch.zeros(3)
    for args, err in (((x[:2], x, m, m), ValueError), ((bf(3, 8), x, m, m), TypeError), ((x, x, m[:2], m), ValueError)):
        with pytest.raises(err):
            ia.layer_norm_bwd(*args)
    lg, s = torch.zeros(2, 3, 9), torch.zeros(2, 3)
    for args, kw, err in (((lg[0], s, 2), {}, ValueError), ((lg, s[:1], 2), {}, ValueError), ((lg, s.double(), 2), {}, TypeError),
                          ((lg, s, 2), dict(finished=torch.zeros(2, 2)), ValueError),
                          ((lg, s, 2), dict(finished=torch.zeros(2, 3)), TypeError), ((lg.double(), s, 2), {}, TypeError)):
        with pytest.raises(err):
            ia.beam_select(*args, **kw)
    par = torch.zeros(2, 3, dtype=torch.int32)
    n = 6 * 2 * 16 * (8 + 4 + 1) * 2
    for args, err in (((torch.zeros(n - 1), par, 6, 2, 16, 8, 4), ValueError), ((torch.zeros(n), par.long(), 6, 2, 16, 8, 4), TypeError),
                      ((torch.zeros(n), par[0], 6, 2, 16, 8, 4), ValueError),
                      ((torch.zeros(n), torch.zeros(4, 3, dtype=torch.int32), 6, 2, 16, 8, 4), ValueError)):
        with pytest.raises(err):
            ia.state_reorder(*args)


def test_binding_refuses_strided_tensors(lib, monkeypatch):
    monkeypatch.setattr(ia, "_place", lambda *named: 0)
    monkeypatch.setattr(ia, "_on", lambda idx, stream: (ia._CURRENT, 0))
    q, k, v, g = seq(N=6)
    with pytest.raises(ValueError, match="contiguous"):
        ia.linear_prefill_fwd(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, g)
    with pytest.raises(ValueError, match="contiguous"):
        ia.layer_norm_fwd(torch.zeros(8, 3).t())


def test_sizes_beyond_an_int_are_refused(lib):
    with pytest.raises(ValueError, match="2\\^31"):
        ia._small("x", 3, 1 << 31)


def test_outputs_may_not_overlap_inputs(lib):
    q, v = torch.zeros(1, 1, 8, 16), torch.zeros(1, 1, 8, 16)
    g = torch.zeros(1)
    with pytest.raises(ValueError, match="overlaps"):
        ia.linear_prefill_fwd(q, q.clone(), v, g, o=v)
    step = [torch.zeros(1, 1, 16) for _ in range(3)]
    with pytest.raises(ValueError, match="overlaps"):
        ia.linear_decode_step(*step, g, torch.zeros(256), o=step[0])
    buf = torch.zeros(9, 16)
    with pytest.raises(ValueError, match="overlaps"):
        ia.layer_norm_fwd(buf[:8], y=buf[1:])
    with pytest.raises(ValueError, match="overlaps"):
        ia.layer_norm_bwd(torch.zeros(8, 16), buf[1:], torch.zeros(8), torch.zeros(8), dx=buf[:8])
    for same in (dict(x=buf, y=buf), dict(x=buf, y=None)):      # in place as a whole: stops only at the CPU tensors
        with pytest.raises(ValueError, match="CUDA"):
            ia.layer_norm_fwd(**same)
