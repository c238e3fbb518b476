"""The embedding's and the head's operators in 64 bits on the CPU, with the
bound on a kernel's error that its roundings allow (element by element).

u = 2^-24 is the relative error of one fp32 rounding, ut that of the element
type (bf16: 2^-8).  A sum of n fp32 terms in any order is off by at most
(n - 1) u times the sum of their absolute values (to first order; the bounds
below take n + 8, which covers second order and the products' own roundings).
"""
import torch

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
UT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def scatter(tokens, grad, vocab, scale, dtype, base=None):
    """(gradient, bound) of the embedding table, float64 [vocab, dim]."""
    t, g = tokens.flatten().long(), grad.reshape(-1, grad.shape[-1]).double()
    ok = (t >= 0) & (t < vocab)
    t, g = t[ok], g[ok]
    out = torch.zeros(vocab, g.shape[1], dtype=torch.float64).index_add_(0, t, g) * scale
    mass = torch.zeros_like(out).index_add_(0, t, g.abs()) * abs(scale)
    count = torch.zeros(vocab, 1, dtype=torch.float64).index_add_(0, t, torch.ones(len(t), 1, dtype=torch.float64))
    if base is not None:
        out = out + base.double()
    err = (count + 8) * U * mass + (UT[dtype] + U) * out.abs() * 1.01
    if base is not None:
        err = torch.where(count > 0, err, torch.zeros_like(err))  # rows without a token stay as they were
    return out, err


def head(hidden, weight, targets, scale, dtype, grad_loss=None, base=None):
    """dict of float64 results and their bounds: loss, lse and, with grad_loss,
    gh and gw; keys name + "_err" hold the bounds."""
    D, V = hidden.shape[-1], weight.shape[0]
    t = targets.flatten().long()
    ok = (t >= 0) & (t < V)
    h = torch.where(ok[:, None], hidden.reshape(-1, D).double(), 0.0)
    w = weight.double().contiguous()
    at = torch.where(ok, t, 0)[:, None]
    z = h @ w.T.contiguous() * scale
    ez = (D + 8) * U * (h.abs() @ w.abs().T.contiguous()) * abs(scale)  # error of a logit
    ezr = ez.max(1).values
    lse = torch.logsumexp(z, 1)
    spread = (z.max(1).values[:, None] - z).clamp(max=100).max(1).values
    # the sum of exponentials: at most 300 additions deep, each exponential
    # off by its argument's roundings (spread u) and a few ulp
    elog = (300 + 2 * spread + 16) * U
    elogr = ezr + elog + 4 * U * lse.abs()
    loss = lse - z.gather(1, at)[:, 0]
    eloss = elogr + ezr + 4 * U * (loss.abs() + lse.abs())
    zero = torch.zeros_like(lse)
    out = dict(lse=torch.where(ok, lse, zero), lse_err=torch.where(ok, elogr, zero),
               loss=torch.where(ok, loss, zero), loss_err=torch.where(ok, eloss, zero))
    if grad_loss is None:
        return out
    g = torch.where(ok, grad_loss.flatten().double(), zero)[:, None] * scale
    p = torch.exp(z - lse[:, None])
    G = p.clone()
    G[torch.arange(len(t), device=t.device), at[:, 0]] -= 1.0
    G = G * g
    # a probability is off by its exponent's error; G is rounded to the
    # element type (bf16) or held in fp32
    eG = g.abs() * p * 1.1 * (ez + elogr[:, None] + (spread[:, None] + 16) * U) + G.abs() * (4 * U + (UT[dtype] if dtype != "f32" else 0.0))
    out["gh"] = G @ w
    out["gh_err"] = eG @ w.abs() + (V + 8) * U * (G.abs() @ w.abs()) + (UT[dtype] + U) * 1.01 * out["gh"].abs()
    out["gw"] = G.T @ h
    if base is not None:
        out["gw"] = out["gw"] + base.double()
    out["gw_err"] = (eG.T @ h.abs() + (len(t) + 8) * U * (G.abs().T @ h.abs()) + (UT[dtype] + U) * 1.01 * out["gw"].abs())
    return out


def check(name, got, want, err):
    """got within err of want everywhere (err also takes the smallest normal
    number: results below it may be flushed)."""
    got = got.double().cpu().reshape(want.shape)
    assert torch.isfinite(got).all(), f"{name}: {int((~torch.isfinite(got)).sum())} values are not finite"
    off = (got - want).abs() - err - 2.0 ** -120
    if (off > 0).any():
        i = int(off.argmax())
        raise AssertionError(f"{name}: {int((off > 0).sum())} of {off.numel()} outside the bound; at {i} got "
                             f"{got.flatten()[i]:.9g}, want {want.flatten()[i]:.9g} +- {err.flatten()[i]:.3g}")
