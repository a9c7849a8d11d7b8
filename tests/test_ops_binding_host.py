"""What the binding of linear attention, layer norm and beam search refuses before the library sees an address: memory
shared between an output and anything else, and sizes that a C int would cut off."""
import pytest
import torch

import ssm_token_mixer_b200 as ia


@pytest.fixture(scope="module", autouse=True)
def lib():
    from ssm_token_mixer_b200 import build
    build.build()
    return ia.load_library()


def refused(call):
    with pytest.raises(ValueError, match="overlaps"):
        call()


def passes(call):
    """Every check of memory is passed: only the CPU tensors stop the call."""
    with pytest.raises(ValueError, match="CUDA"):
        call()


B, H, N, DK, DV = 2, 3, 5, 8, 4
FP = torch.float32


def pool(*sizes, dtype=FP):
    """Tensors laid one after the other in one buffer, on 16-byte boundaries, and the buffer."""
    total = sum(torch.Size(s).numel() + 3 for s in sizes)
    buf, at, out = torch.zeros(total + 64, dtype=dtype), 0, []
    for s in sizes:
        n = torch.Size(s).numel()
        out.append(buf[at:at + n].view(s))
        at += -(-n // 4) * 4
    return buf, out


def test_linear_prefill():
    buf, (q, k, v, g, s, o) = pool((B, H, N, DK), (B, H, N, DK), (B, H, N, DV), (H,), (B, H, DK, DV), (B, H, N, DV))
    passes(lambda: ia.linear_prefill_fwd(q, k, v, g, state_in=s, o=o))
    n = o.numel()
    for t in (q, k, v, s):
        last = t.storage_offset() + t.numel() - 1     # only one value is shared
        refused(lambda: ia.linear_prefill_fwd(q, k, v, g, state_in=s, o=buf[last:last + n].view_as(o)))
    wide = g.storage_offset()
    refused(lambda: ia.linear_prefill_fwd(q, k, v, g, o=buf[wide:wide + n].view_as(o)))
    for t in (q, k, v, g, s, o):
        refused(lambda: ia.linear_prefill_fwd(q, k, v, g, state_in=s, o=o, workspace=t.view(-1)))


def test_linear_training_step():
    buf, (q, k, v, dO, g) = pool((B, H, N, DK), (B, H, N, DK), (B, H, N, DV), (B, H, N, DV), (H,))
    passes(lambda: ia.linear_fwd_bwd(q, k, v, g, dO, workspace=buf[-64:]))
    for t in (q, k, v, dO, g):
        refused(lambda: ia.linear_fwd_bwd(q, k, v, g, dO, workspace=t.view(-1)))


def test_linear_decode(monkeypatch):
    monkeypatch.setenv("IA_INJECT_LAUNCH_FAILURE", "1")   # what passes every check ends in the library, without a launch
    monkeypatch.setattr(ia, "_place", lambda *named: 0)   # (the state is looked at after the tensors' device)
    monkeypatch.setattr(ia, "_on", lambda idx, stream: (ia._CURRENT, 0))

    def passes(call):
        with pytest.raises(ia.IAError) as e:
            call()
        assert e.value.status == 4

    n = B * H * DK * DV
    buf, (q, k, v, g, s, so, o) = pool((B, H, DK), (B, H, DK), (B, H, DV), (H,), (n,), (n,), (B, H, DV))
    par = torch.zeros(1, B, dtype=torch.int32)
    passes(lambda: ia.linear_decode_step(q, k, v, g, s, o=o))
    passes(lambda: ia.linear_decode_step(q, k, v, g, s, state_out=s))             # in place
    passes(lambda: ia.linear_decode_step(q, k, v, g, s, state_out=so, parents=par, o=o))
    for t in (q, k, v, g):
        at = t.storage_offset()
        refused(lambda: ia.linear_decode_step(q, k, v, g, s, state_out=buf[at:at + n]))
        refused(lambda: ia.linear_decode_step(q, k, v, g, buf[at:at + n]))        # the state that is updated in place
        refused(lambda: ia.linear_decode_step(q, k, v, g, s, o=buf[at:at + o.numel()].view_as(o)))
    mine = so.view(torch.int32)[5:5 + B].view(1, B)
    refused(lambda: ia.linear_decode_step(q, k, v, g, s, state_out=so, parents=mine))
    theirs = o.view(-1).view(torch.int32)[:B].view(1, B)
    refused(lambda: ia.linear_decode_step(q, k, v, g, s, state_out=so, parents=theirs, o=o))


def test_layer_norm():
    buf, (x, dy, w, b, m, r) = pool((6, 16), (6, 16), (16,), (16,), (6,), (6,))
    passes(lambda: ia.layer_norm_fwd(x, w, b, y=x))
    passes(lambda: ia.layer_norm_bwd(dy, x, m, r, w, dx=dy))
    passes(lambda: ia.layer_norm_bwd(dy, x, m, r, w, dx=x, workspace=buf[-64:]))
    n = x.numel()
    for t in (w, b):
        at = t.storage_offset() + 15 - n + 1
        refused(lambda: ia.layer_norm_fwd(torch.zeros(6, 16), w, b, y=buf[at:at + n].view(6, 16)))
    for t in (w, m, r):
        at = t.storage_offset() + t.numel() - n
        refused(lambda: ia.layer_norm_bwd(torch.zeros(6, 16), torch.zeros(6, 16), m, r, w, dx=buf[at:at + n].view(6, 16)))
    for t in (x, dy, w, m, r):
        refused(lambda: ia.layer_norm_bwd(dy, x, m, r, w, workspace=t.view(-1)))
    dx = torch.zeros(6, 16)
    refused(lambda: ia.layer_norm_bwd(dy, x, m, r, w, dx=dx, workspace=dx))


def test_beam_and_reorder():
    _, (x, s) = pool((2, 3, 9), (2, 3))
    fin = torch.zeros(2, 3, dtype=torch.uint8)
    passes(lambda: ia.beam_select(x, s, 2, finished=fin, workspace=torch.zeros(8, dtype=torch.uint8)))
    for t in (x, s, fin):
        refused(lambda: ia.beam_select(x, s, 2, finished=fin, workspace=t.view(-1)))
    st = torch.zeros(2 * H * DK * DV)
    par = torch.zeros(1, 2, dtype=torch.int32)
    passes(lambda: ia.linear_state_reorder(st, par, 2, H, DK, DV, out=st))
    out = torch.zeros_like(st)
    refused(lambda: ia.linear_state_reorder(st, out.view(torch.int32)[3:5].view(1, 2), 2, H, DK, DV, out=out))


BIG = 2**32   # as a C int: 0


def test_sizes_that_a_c_int_would_cut_off():
    par = torch.zeros(1, 2, dtype=torch.int32)
    st = torch.zeros(2 * H * DK * DV)
    x, s = torch.zeros(1, 2, 9), torch.zeros(1, 2)
    fin = torch.zeros(1, 2, dtype=torch.bool)
    for call in (lambda: ia.linear_state_bytes(BIG + 1, H, DK, DV), lambda: ia.linear_path(1, H, BIG + 5, DK, DV, "bf16"),
                 lambda: ia.linear_prefill_workspace_bytes(1, H, 5, BIG + DK, DV, "f32"),
                 lambda: ia.linear_fwd_bwd_workspace_bytes(1, BIG + H, 5, DK, DV, "f32"),
                 lambda: ia.linear_prefill_segments(1, H, BIG + 5, DK, DV, "f32"),
                 lambda: ia.linear_fwd_bwd_segments(1, H, 5, DK, BIG + DV, "f32"),
                 lambda: ia.linear_state_reorder(st, par, BIG + 2, H, DK, DV),
                 lambda: ia.state_reorder(st, par, 2, H, BIG + 1, DK, DV),
                 lambda: ia.layer_norm_bwd_workspace_bytes(4, BIG + 8, "f32"),
                 lambda: ia.beam_select_workspace_bytes(1, 2, BIG + 9, 2, "f32"),
                 lambda: ia.beam_select(x, s, BIG + 2), lambda: ia.beam_select(x, s, 2, finished=fin, end_token=BIG + 3),
                 lambda: ia.beam_select(x, s, 2, finished=fin, end_token=-BIG)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert ia.linear_state_bytes(2, H, DK, DV) == st.numel() * 4
