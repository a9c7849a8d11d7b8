"""Plain fp64 forms of linear attention, layer norm and beam search, written
from their definitions token by token and row by row (test infrastructure),
with the bounds that the kernels' roundings give.

Bounds.  A sum of n products in fp32 is off by at most n u sum|terms|, u =
2^-24 (and the smaller second-order terms), whatever its order.  ``magnitude``
is that sum of absolute terms, from the same recurrence on absolute values.
For the tensor-core path they leave room for one rounding of each decayed
score and each entry of the entering state to bf16 (2^-8 each, on disjoint
groups of terms: 2^-8 magnitude) and for weighted values that reach the state
in two bf16 parts (2^-16).  The kernels keep more of both, which
test_gpu_linear_accuracy.py and test_gpu_linear_state.py hold them to.  A bf16
result adds 2^-8 of itself.
"""
import torch

U = 2.0 ** -24
BF = 2.0 ** -8


def recurrence(x, y, z, log_decay, state=None, reverse=False):
    """out_t = x_t S_t with S_t = lambda S_(t-1) + y_t z_t^T in fp64, and the last S."""
    x, y, z = x.double(), y.double(), z.double()
    lam = torch.exp(log_decay.double())[None, :, None, None]
    S = torch.zeros(*y.shape[:2], y.shape[3], z.shape[3], dtype=torch.float64, device=x.device)
    if state is not None:
        S = S + state.double().view_as(S)
    out = torch.empty(*x.shape[:3], z.shape[3], dtype=torch.float64, device=x.device)
    N = x.shape[2]
    for t in (range(N - 1, -1, -1) if reverse else range(N)):
        S = lam * S + y[:, :, t, :, None] * z[:, :, t, None, :]
        out[:, :, t] = torch.einsum("bhi,bhij->bhj", x[:, :, t], S)
    return out, S


def linear_bounds(x, y, z, log_decay, scale, tc, state=None, reverse=False):
    """(out, its elementwise bound, state, its bound) for one direction."""
    out, S = recurrence(x, y, z, log_decay, state, reverse)
    mag, Smag = recurrence(x.abs(), y.abs(), z.abs(), log_decay, None if state is None else state.abs(), reverse)
    # roundings on the way of one term: the products over dx, the chunk's sum, the decays
    # (|exponent| u e^-|exponent| <= u / 2 each, their weights and expf's 2 ulp) and one multiply-add per chunk
    n = x.shape[3] + 128 + 2 * (x.shape[2] // 32 + 1) + 16
    u = n * U + (BF if tc else 0.0)
    out, mag = out * scale, mag * abs(scale)
    err = u * mag
    if x.dtype == torch.bfloat16:
        err = err + BF * (out.abs() + err)
    su = (n + 0.0) * U + (2.0 ** -16 if tc else 0.0)
    return out, err + 1e-30, S, su * Smag + 1e-30


def layer_norm(x, weight, bias, eps):
    x = x.double()
    mean = x.mean(-1)
    c = x - mean[..., None]
    rstd = 1.0 / torch.sqrt(c.square().mean(-1) + eps)
    hat = c * rstd[..., None]
    y = hat * (1.0 if weight is None else weight.double()) + (0.0 if bias is None else bias.double())
    return y, mean, rstd, hat


def layer_norm_grads(dy, x, weight, eps):
    dy = dy.double()
    _, _, rstd, hat = layer_norm(x, None, None, eps)
    g = dy if weight is None else dy * weight.double()
    dx = rstd[..., None] * (g - g.mean(-1, keepdim=True) - hat * (g * hat).mean(-1, keepdim=True))
    flat = (-1, x.shape[-1])
    return dx, (dy * hat).reshape(flat).sum(0), dy.reshape(flat).sum(0)


def beam_select(logits, scores, K, finished=None, end_token=0):
    """Request by request: every candidate with its exact score, sorted by (score down, beam, token)."""
    x, s = logits.double().cpu(), scores.double().cpu()
    fin = None if finished is None else finished.cpu().bool()
    out = []
    for g in range(x.shape[0]):
        cand = []
        for w in range(x.shape[1]):
            if not torch.isfinite(s[g, w]):
                continue
            if fin is not None and fin[g, w]:
                cand.append((-float(s[g, w]), w, end_token))
                continue
            row = x[g, w]
            if torch.isnan(row).any() or (row == float("inf")).any() or row.max() == -float("inf"):
                continue
            lse = row.max() + torch.log(torch.exp(row - row.max()).sum())
            best = torch.sort(row, descending=True, stable=True)
            for v, t in zip(best.values[:K].tolist(), best.indices[:K].tolist()):
                if v > -float("inf"):
                    cand.append((-(float(s[g, w]) + (v - float(lse))), w, t))
        cand.sort()
        cand = cand[:K] + [(float("inf"), -1, -1)] * (K - len(cand))
        out.append(cand)
    f = lambda i, sign, dt: torch.tensor([[sign * c[i] for c in row] for row in out], dtype=dt)  # noqa: E731
    return f(0, -1, torch.float64), f(1, 1, torch.int32), f(2, 1, torch.int32)
