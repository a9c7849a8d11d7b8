"""Cases of the layer's linear-attention mixer, its layer norm and beam search, each in a plain form and as a call
of the library.

The plain form (``own`` false) is written with elementary torch operations in fp32, or fp64 where fp32 would decide
a close comparison differently, and rounds once at the end.  With ``own`` true the same inputs go through
``ssm_token_mixer_b200``.

Kinds of case:
  prefill   causal linear attention with one decay per head over a prompt, o and the state after it
  train     the same from a zero state, with the gradients of q, k and v
  decode    one token of it per sequence, optionally reading its state through the beams' parents
  norm      layer norm: y and the row statistics; with "bwd" also dx, dweight and dbias
  beam      the best K continuations over beams and vocabulary; with "H" also the reordering of the layer's states
"""
import math

import torch

own = False

CHUNK = 64   # tokens per block of the plain form's products


def listed():
    return [
        # a prompt through a layer of 12 heads of 64 (the 125M layer's shape)
        dict(name="prefill_12x64", kind="prefill", dtype="bf16", B=8, H=12, N=2048, dk=64, dv=64, cont=False),
        # one long prompt continued from an earlier state, its length a multiple of nothing (the 1.3B layer's shape)
        dict(name="prefill_long_ragged", kind="prefill", dtype="bf16", B=1, H=16, N=7001, dk=128, dv=128, cont=True),
        # fp32 inputs and head widths that are no power of two, as tests and small models have them
        dict(name="prefill_f32_small", kind="prefill", dtype="f32", B=2, H=4, N=300, dk=48, dv=80, cont=False),
        # a training step of 16 heads of 64 (the 350M layer's shape)
        dict(name="train_16x64", kind="train", dtype="bf16", B=8, H=16, N=2048, dk=64, dv=64),
        # a training step on a short ragged batch with wide heads
        dict(name="train_ragged_128", kind="train", dtype="bf16", B=3, H=5, N=777, dk=128, dv=128),
        # one sequence, one token: the latency of a decode step
        dict(name="decode_1", kind="decode", dtype="bf16", B=1, H=16, dk=128, dv=128, W=0),
        # 16 requests of 4 beams: each beam reads its parent's state and writes its own
        dict(name="decode_beams_64", kind="decode", dtype="bf16", B=64, H=16, dk=128, dv=128, W=4),
        # the norm of a training step, 8 x 2048 tokens of width 1024
        dict(name="norm_train_1024", kind="norm", dtype="bf16", rows=16384, D=1024, bwd=True),
        # fp32 rows of an odd width
        dict(name="norm_train_f32_777", kind="norm", dtype="f32", rows=5003, D=777, bwd=True),
        # one request with four beams: the latency of a selection
        dict(name="beam_1x4", kind="beam", dtype="f32", G=1, W=4, V=32000, K=4, H=0),
        # a full serving batch, twice as many candidates as beams, an odd vocabulary
        dict(name="beam_64x8", kind="beam", dtype="bf16", G=64, W=8, V=50257, K=16, H=0),
        # selection, then the layer's recurrent states follow their parents (16 heads, d = 128, M = 64)
        dict(name="beam_step_16x4", kind="beam", dtype="bf16", G=16, W=4, V=32000, K=4, H=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "train", "train", "decode", "norm", "norm", "beam", "beam"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    if kind in ("prefill", "train"):
        wide = dtype == "bf16"
        dk, dv = (rng.choice([64, 128]), rng.choice([64, 128])) if wide else (rng.randint(8, 128), rng.randint(8, 128))
        N = _log_int(rng, 1, 8192)
        most = (8 * 16 * 2048 * 64 if wide else 1 << 20) // max(dk, dv)   # tokens x heads
        H = rng.randint(1, 24)
        N = max(1, min(N, most // H))
        B = _log_int(rng, 1, max(1, min(16, most // (H * N))))
        c = dict(kind=kind, dtype=dtype, B=B, H=H, N=N, dk=dk, dv=dv)
        if kind == "prefill":
            c["cont"] = rng.random() < 0.5
        return c
    if kind == "decode":
        W = rng.choice([0, 0, 2, 3, 4, 5, 8])
        G = _log_int(rng, 1, 64 // max(1, W))
        dk, dv = (rng.choice([64, 128]), rng.choice([64, 128])) if dtype == "bf16" else (rng.randint(8, 128), rng.randint(8, 128))
        return dict(kind=kind, dtype=dtype, B=G * max(1, W), H=rng.randint(1, 16), dk=dk, dv=dv, W=W)
    if kind == "norm":
        D = rng.choice([64, 128, 256, 768, 1024, 2048, 4096, 8192, _log_int(rng, 17, 9000), _log_int(rng, 17, 9000)])
        return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 1, min(131072, (1 << 24) // D)), D=D, bwd=rng.random() < 0.6)
    W = rng.choice([1, 2, 3, 4, 5, 8, 16])
    G = _log_int(rng, 1, 512 // W)
    V = _log_int(rng, 1000, 131072)
    while G > 1 and G * W * V > 512 * 50257:
        G //= 2
    K = rng.choice([W, 2 * W, rng.randint(1, 2 * W)])
    H = rng.choice([0, 0, 8, 12, 16]) if G * W <= 64 else 0
    return dict(kind=kind, dtype=dtype, G=G, W=W, V=V, K=W if H else K, H=H)


STATE_M, STATE_D = 64, 128   # modes and head width of the layer's states in the beam cases


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    t = _type(case)

    def normal(*shape, std=1.0, mean=0.0, dtype=t):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case=case)
    kind = case["kind"]
    if kind in ("prefill", "train", "decode"):
        H = case["H"]
        # decays 1 - 2^-u from about 0.3 forgotten per token to almost nothing over a long prompt
        s["log_decay"] = torch.log1p(-torch.exp2(-uniform(H, lo=1.5, hi=12.0).double())).float()
        lead = (case["B"], H) if kind == "decode" else (case["B"], H, case["N"])
        s["q"], s["k"], s["v"] = normal(*lead, case["dk"]), normal(*lead, case["dk"]), normal(*lead, case["dv"])
        if kind == "train":
            s["dO"] = normal(*lead, case["dv"])
        if kind == "decode" or case.get("cont"):
            s["state"] = normal(case["B"], H, case["dk"], case["dv"], std=4.0, dtype=torch.float32).reshape(-1)
        if case.get("W"):
            W = case["W"]
            s["parents"] = torch.randint(0, W, (case["B"] // W, W), generator=g, device="cuda", dtype=torch.int32)
            s["other"] = torch.empty_like(s["state"])   # the second of the two state buffers
    elif kind == "norm":
        s["x"] = normal(case["rows"], case["D"], std=1.5, mean=0.4)
        s["weight"] = normal(case["D"], std=0.3, mean=1.0, dtype=torch.float32)
        s["bias"] = normal(case["D"], std=0.2, dtype=torch.float32)
        if case["bwd"]:
            s["dy"] = normal(case["rows"], case["D"])
    else:
        G, W, V = case["G"], case["W"], case["V"]
        s["logits"] = normal(G, W, V, std=2.5)
        s["logits"][:, :, V // 2::97] = -math.inf   # suppressed tokens
        s["scores"] = -torch.cumsum(uniform(G, W, lo=0.0, hi=2.0), 1) - 20.0
        s["finished"] = uniform(G, W) < 0.1
        if W > 1:   # some requests run with fewer live beams
            s["scores"][uniform(G) < 0.1, W - 1] = -math.inf
        if case["H"]:
            n = G * W * case["H"] * STATE_M * (2 * STATE_D + 1) * 2
            s["state"], s["other"] = normal(n, dtype=torch.float32), torch.empty(n, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _blocks(x, n):
    """[.., N, d] in fp32, filled up with zeros to n blocks of CHUNK tokens: [.., n, CHUNK, d]."""
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, n * CHUNK - x.shape[-2]))
    return x.unflatten(-2, (n, CHUNK))


def _decayed(x, y, z, log_decay, state=None):
    """sum over s <= t of lambda^(t-s) (x_t . y_s) z_s, plus lambda^(t+1) x_t state."""
    N = x.shape[-2]
    n = -(-N // CHUNK)
    x, y, z = _blocks(x, n), _blocks(y, n), _blocks(z, n)
    g = log_decay.double()[:, None, None]
    i = torch.arange(CHUNK, device=x.device, dtype=torch.float64)
    far = i[:, None] - i[None, :]
    within = torch.where(far >= 0, torch.exp(g * far.clamp(min=0)), 0.0).float()          # [H,C,C]
    tail = torch.exp(g * (CHUNK - 1 - i)[None, :, None]).float()[:, None]                  # [H,1,C,1]
    head = torch.exp(g * (i + 1)[None, :, None]).float()[:, None]
    c = torch.arange(n, device=x.device, dtype=torch.float64)
    gap = c[:, None] - 1 - c[None, :]
    across = torch.where(gap >= 0, torch.exp(g * CHUNK * gap.clamp(min=0)), 0.0).float()  # [H,n,n]
    local = (y * tail).transpose(-1, -2) @ z                                              # [B,H,n,dx,dz]
    entering = (across @ local.flatten(-2)).unflatten(-1, local.shape[-2:])               # [B,H,n,dx,dz]
    if state is not None:
        entering = entering + torch.exp(g * CHUNK * c[None, :, None]).float()[..., None] * state[:, :, None]
    out = ((x @ y.transpose(-1, -2)) * within[:, None]) @ z + (x * head) @ entering
    return out.flatten(-3, -2)[..., :N, :]


def _last_state(y, z, log_decay, state):
    """The state after the last token, by one weighted product over all tokens (no division by small decays)."""
    N = y.shape[-2]
    g = log_decay.double()[:, None, None]
    w = torch.exp(g * (N - 1 - torch.arange(N, device=y.device, dtype=torch.float64))[None, :, None]).float()
    s = (y.float() * w).transpose(-1, -2) @ z.float()
    return s if state is None else s + torch.exp(g * N).float() * state


def _plain_prefill(s):
    c = s["case"]
    state = s["state"].view(c["B"], c["H"], c["dk"], c["dv"]) if c["cont"] else None
    o = _decayed(s["q"], s["k"], s["v"], s["log_decay"], state)
    return {"o": (o * c["dk"] ** -0.5).to(s["q"].dtype), "state": _last_state(s["k"], s["v"], s["log_decay"], state).reshape(-1)}


def _plain_train(s):
    q, k, v, dO, g, t = s["q"], s["k"], s["v"], s["dO"], s["log_decay"], s["q"].dtype
    scale = s["case"]["dk"] ** -0.5
    back = [x.flip(-2) for x in (q, k, v, dO)]
    o = _decayed(q, k, v, g)
    dq = _decayed(dO, v, k, g)
    dk = _decayed(back[2], back[3], back[0], g).flip(-2)
    dv = _decayed(back[1], back[0], back[3], g).flip(-2)
    return {n: (x * scale).to(t) for n, x in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv))}


def _plain_decode(s):
    c = s["case"]
    state = s["state"].view(c["B"], c["H"], c["dk"], c["dv"])
    if c["W"]:
        rows = torch.arange(c["B"] // c["W"], device=state.device)[:, None] * c["W"] + s["parents"]
        state = state[rows.reshape(-1).long()]
    state = torch.exp(s["log_decay"])[:, None, None] * state + s["k"].float()[..., :, None] * s["v"].float()[..., None, :]
    o = (s["q"].float()[..., None, :] @ state)[..., 0, :] * c["dk"] ** -0.5
    kept = s["other"] if c["W"] else s["state"]
    kept.copy_(state.reshape(-1))
    return {"o": o.to(s["q"].dtype), "state": kept}


def _plain_norm(s):
    eps = 1e-5
    x, t = s["x"].float(), s["x"].dtype
    mean = x.mean(-1)
    centred = x - mean[:, None]
    rstd = (centred.square().mean(-1) + eps).rsqrt()
    hat = centred * rstd[:, None]
    out = {"y": (hat * s["weight"] + s["bias"]).to(t), "mean": mean, "rstd": rstd}
    if s["case"]["bwd"]:
        dy = s["dy"].float()
        d = dy * s["weight"]
        dx = rstd[:, None] * (d - d.mean(-1, keepdim=True) - hat * (d * hat).mean(-1, keepdim=True))
        out |= {"dx": dx.to(t), "dweight": (dy * hat).sum(0), "dbias": dy.sum(0)}
    return out


def _candidates(s):
    """The score of every (beam, token) in fp64, [G, W*V]: beam score + log softmax; -inf for what may not be chosen."""
    c = s["case"]
    x, score = s["logits"].double(), s["scores"].double()[..., None]
    top = x.amax(-1, keepdim=True)
    total = score + (x - top - torch.exp(x - top).sum(-1, keepdim=True).log())
    total = torch.where(torch.isnan(total) | torch.isinf(score), -math.inf, total)
    # a finished beam has one continuation: the end token, at its own score
    end = torch.where(torch.arange(c["V"], device=x.device) == END, score, -math.inf)
    return torch.where(s["finished"][..., None], end, total).flatten(1)


END = 2   # the end token's index


def _plain_beam(s):
    c = s["case"]
    best, at = torch.sort(_candidates(s), dim=1, descending=True, stable=True)
    best, at = best[:, :c["K"]], at[:, :c["K"]]
    none = torch.isinf(best)
    out = {"scores": best.float(), "parents": torch.where(none, -1, at // c["V"]).int(),
           "tokens": torch.where(none, -1, at % c["V"]).int()}
    if c["H"]:
        B = c["G"] * c["W"]
        rows = (torch.arange(c["G"], device=at.device)[:, None] * c["W"] + out["parents"].clamp(min=0)).reshape(-1).long()
        gone = (out["parents"] < 0).reshape(-1)
        n = B * c["H"] * STATE_M
        sizes = [n * STATE_D * 2, n * STATE_D * 2, n * 2]   # U, Gamma and eta, each with the sequence first
        parts = [torch.where(gone[:, None], 0.0, p.view(B, -1)[rows]) for p in s["state"].split(sizes)]
        out["state"] = torch.cat([p.reshape(-1) for p in parts], out=s["other"])
    return out


def run(state):
    s, c = state, state["case"]
    kind = c["kind"]
    if not own:
        return {"prefill": _plain_prefill, "train": _plain_train, "decode": _plain_decode, "norm": _plain_norm,
                "beam": _plain_beam}[kind](s)
    import ssm_token_mixer_b200 as ia
    if kind == "prefill":
        r = ia.linear_prefill_fwd(s["q"], s["k"], s["v"], s["log_decay"], state_in=s.get("state"), want_state=True)
        return {"o": r["o"], "state": r["state"]}
    if kind == "train":
        r = ia.linear_fwd_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["dO"])
        return {n: r[n] for n in ("o", "dq", "dk", "dv")}
    if kind == "decode":
        r = ia.linear_decode_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], parents=s.get("parents"),
                                  state_out=s.get("other"))
        return {"o": r["o"], "state": r["state"]}
    if kind == "norm":
        r = ia.layer_norm_fwd(s["x"], s["weight"], s["bias"])
        out = {n: r[n] for n in ("y", "mean", "rstd")}
        if c["bwd"]:
            b = ia.layer_norm_bwd(s["dy"], s["x"], r["mean"], r["rstd"], s["weight"])
            out |= {n: b[n] for n in ("dx", "dweight", "dbias")}
        return out
    r = ia.beam_select(s["logits"], s["scores"], c["K"], finished=s["finished"], end_token=END)
    out = {n: r[n] for n in ("scores", "parents", "tokens")}
    if c["H"]:
        out["state"] = ia.state_reorder(s["state"], r["parents"], c["G"] * c["W"], c["H"], STATE_M, STATE_D, STATE_D,
                                        out=s["other"])
    return out


# ------------------------------------------------------------------- the work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    kind = case["kind"]
    if kind in ("prefill", "train"):
        T, dk, dv = case["B"] * case["H"] * case["N"], case["dk"], case["dv"]
        state = case["B"] * case["H"] * dk * dv * 4
        if kind == "prefill":   # q, k, v in, o and the state out; the recurrence's update and read
            return {"bytes": e * T * (2 * dk + 2 * dv) + state * (2 if case["cont"] else 1) + 4 * case["H"], "flops": 4 * T * dk * dv}
        # q, k, v, dO in, o, dq, dk, dv out; two recurrences, four reads
        return {"bytes": e * T * (4 * dk + 4 * dv) + 4 * case["H"], "flops": 12 * T * dk * dv}
    if kind == "decode":
        BH, dk, dv, W = case["B"] * case["H"], case["dk"], case["dv"], case["W"]
        read = 1 - (1 - 1 / W) ** W if W else 1.0   # the share of the states that some beam follows, on average
        return {"bytes": 4 * BH * dk * dv * (1 + read) + e * BH * (2 * dk + 2 * dv), "flops": 5 * BH * dk * dv}
    if kind == "norm":
        n, D = case["rows"] * case["D"], case["D"]
        if not case["bwd"]:
            return {"bytes": 2 * n * e + 8 * case["rows"] + 8 * D, "flops": 8 * n}
        return {"bytes": 4 * n * e + 8 * case["rows"] + 16 * D, "flops": 20 * n}
    n = case["G"] * case["W"] * case["V"]
    b = n * e + 5 * case["G"] * case["W"] + 12 * case["G"] * case["K"]
    if case["H"]:   # a state read per beam that is followed, a state written per beam
        W = case["W"]
        b += case["G"] * W * case["H"] * STATE_M * (2 * STATE_D + 1) * 8 * (2 - (1 - 1 / W) ** W)
    return {"bytes": b, "flops": 4 * n}


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    def recurrence(x, y, z, log_decay, state=None, reverse=False):
        """S_t = lambda S_(t-1) + y_t z_t^T and x_t S_t, token after token (from the last one back with reverse)."""
        x, y, z = (t.double().movedim(2, 0).contiguous() for t in (x, y, z))
        lam = torch.exp(log_decay.double())[None, :, None, None]
        S = torch.zeros(*y.shape[1:], z.shape[-1], dtype=torch.float64, device=x.device) if state is None else state.double().clone()
        out = torch.empty(*x.shape[:-1], z.shape[-1], dtype=torch.float64, device=x.device)
        for t in (range(len(x) - 1, -1, -1) if reverse else range(len(x))):
            S.mul_(lam).add_(y[t].unsqueeze(-1) * z[t].unsqueeze(-2))
            torch.matmul(x[t].unsqueeze(-2), S, out=out[t].unsqueeze(-2))
        return out.movedim(0, 2), S

    s = prepare(case, seed)
    kind = case["kind"]
    scale = case["dk"] ** -0.5 if "dk" in case else 0.0
    if kind == "prefill":
        state = s["state"].view(case["B"], case["H"], case["dk"], case["dv"]) if case["cont"] else None
        o, S = recurrence(s["q"], s["k"], s["v"], s["log_decay"], state)
        return {"o": o * scale, "state": S.reshape(-1)}
    if kind == "train":
        q, k, v, dO, g = s["q"], s["k"], s["v"], s["dO"], s["log_decay"]
        return {"o": recurrence(q, k, v, g)[0] * scale, "dq": recurrence(dO, v, k, g)[0] * scale,
                "dk": recurrence(v, dO, q, g, reverse=True)[0] * scale, "dv": recurrence(k, q, dO, g, reverse=True)[0] * scale}
    if kind == "decode":
        state = s["state"].view(case["B"], case["H"], case["dk"], case["dv"]).double()
        if case["W"]:
            at = s["parents"].long() + case["W"] * torch.arange(len(s["parents"]), device="cuda").unsqueeze(1)
            state = state.index_select(0, at.flatten())
        S = torch.einsum("h,bhij->bhij", s["log_decay"].double().exp(), state)
        S += torch.einsum("bhi,bhj->bhij", s["k"].double(), s["v"].double())
        return {"o": torch.einsum("bhi,bhij->bhj", s["q"].double(), S) * scale, "state": S.reshape(-1)}
    if kind == "norm":
        x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
        mean = x.sum(1) / case["D"]
        rstd = 1 / torch.sqrt((x * x).sum(1) / case["D"] - mean * mean + 1e-5)
        hat = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
        out = {"y": hat * w + b, "mean": mean, "rstd": rstd}
        if case["bwd"]:
            dy = s["dy"].double()
            a = (dy * w).sum(1, keepdim=True) / case["D"]
            c = (dy * w * hat).sum(1, keepdim=True) / case["D"]
            out |= {"dx": (dy * w - a - hat * c) * rstd.unsqueeze(1), "dweight": torch.einsum("rd,rd->d", dy, hat), "dbias": dy.sum(0)}
        return out
    total = []
    for b in range(case["G"]):   # request by request, its K best scores
        p = torch.log_softmax(s["logits"][b].double(), -1) + s["scores"][b].double().unsqueeze(1)
        p[s["finished"][b]] = -math.inf
        p[:, END] = torch.where(s["finished"][b], s["scores"][b].double(), p[:, END])
        p[torch.isneginf(s["scores"][b])] = -math.inf
        total.append(torch.topk(p.flatten(), case["K"]).values)
    return {"scores": torch.stack(total), "parents": None, "tokens": None, "state": None}
