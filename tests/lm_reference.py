"""Plain float64 forms of the language-model operators, for the tests: written
from the definitions, on the CPU, with element-wise error bounds beside them.

U = 2^-8 is half a step of bfloat16 relative to the value, E = 2^-24 of fp32.
"""
import math

import torch

U = torch.finfo(torch.bfloat16).eps / 2
E = torch.finfo(torch.float32).eps / 2


def f64(t):
    return t.detach().cpu().double()


def contraction_error(n):
    """Relative error, against the sum of the products' magnitudes, of an fp32
    accumulation of n exact products in groups of 16: one step of at most a
    whole ulp (2 E, truncation included) for each group and one for the end."""
    return (n // 16 + 4) * 2 * E


# ------------------------------------------------------------------- rotary

def rotate(x, heads, head_dim, freqs, pos, interleaved, scale, inverse):
    """x [T, heads * head_dim] float64 rotated, and the bound's pair magnitudes."""
    T, rot = x.shape[0], 2 * freqs.numel()
    y, mag = x.reshape(T, heads, head_dim).clone(), torch.zeros(T, heads, head_dim).double()
    turns = pos.double()[:, None] * freqs[None]
    ang = (turns - turns.round()) * (2 * math.pi) * (-1 if inverse else 1)
    c, s = scale * ang.cos()[:, None], scale * ang.sin()[:, None]
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    mag[..., a] = mag[..., b] = abs(scale) * (u.abs() + v.abs())
    return y.reshape(T, -1), mag.reshape(T, -1)


# ------------------------------------------------------------ cross entropy

def cross_entropy(z, w, targets, dloss=None, gscale=1.0):
    """z [T,d], w [V,d] float64; returns a dict of float64 results and bounds."""
    T, d = z.shape
    V = w.shape[0]
    logits = z @ w.T
    lse = torch.logsumexp(logits, 1)
    ok = (targets >= 0) & (targets < V)
    at = torch.where(ok, targets, torch.zeros_like(targets))
    loss = torch.where(ok, lse - logits.gather(1, at[:, None]).squeeze(1), torch.zeros_like(lse))
    up = (torch.ones(T, dtype=torch.float64) if dloss is None else dloss.double()) * gscale
    up = torch.where(ok, up, torch.zeros_like(up))
    p = torch.exp(logits - lse[:, None])
    onehot = torch.zeros_like(p)
    onehot[ok, at[ok]] = 1.0
    g = (p - onehot) * up[:, None]
    dz, dw = g @ w, g.T @ z
    # a logit is off by `le`, so the log-sum-exp too (plus its own few fp32 steps)
    le = contraction_error(d) * (z.abs() @ w.abs().T).amax(1)
    lse_tol = le + (64 * E) * (1 + lse.abs() + logits.abs().amax(1))
    # p's relative error follows from both exponents, g is then off by p's part and a rounding
    g_err = (p * (le + lse_tol)[:, None] + 8 * E * (p + onehot)) * up.abs()[:, None]
    gw = g.abs() @ w.abs()
    dz_tol = U * dz.abs() + (U + contraction_error(V)) * gw + (1 + U) * (g_err @ w.abs())
    gz = g.abs().T @ z.abs()
    # both bf16 halves of g leave U * U of it; fp32 sums over T in two halves
    dw_tol = (U * U + 2 * contraction_error(T)) * gz + g_err.T @ z.abs()
    n = int(ok.sum())
    return {"loss": loss, "lse": lse, "dZ": dz, "dW": dw, "loss_tol": lse_tol + le, "lse_tol": lse_tol,
            "dZ_tol": dz_tol, "dW_tol": dw_tol, "count": n,
            "mean": float(loss.sum()) / n if n else 0.0}


def within(got, ref, tol, what):
    got, err = f64(got), None
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what + ": NaN"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), what + ": infinities"
    err = (got - ref).abs()[~inf]
    excess = err - tol[~inf]
    if excess.numel():
        i = int(excess.argmax())
        assert float(excess.max()) <= 0, "%s: off by %.3g, allowed %.3g (value %.3g)" % (
            what, float(err[i]), float(tol[~inf][i]), float(ref[~inf][i]))
