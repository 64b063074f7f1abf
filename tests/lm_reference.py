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


# ---------------------------------------------------------------- attention

def attention(q, k, v, do, heads, kv_heads, hd, cu_q, cu_k, causal, window, scale):
    """Float64 attention and gradients of packed sequences, with bounds.

    Roundings counted: S is off by its fp32 accumulation (`se`), so a probability
    by the relative amount `pe` (twice: numerator and sum), plus 2^-22 of the
    exponential; P is rounded to bf16 before P V and P^T dO, dS before dS K and
    dS^T Q, and every result once more.  Probabilities are formed against a
    maximum at most 2^8 stale, which costs bf16 nothing (same relative step)."""
    G, f = heads // kv_heads, lambda t: torch.zeros_like(t)
    o, o_t, dq, dq_t = f(q), f(q), f(q), f(q)
    dk, dk_t, dv, dv_t = f(k), f(k), f(v), f(v)
    lse = torch.full((heads, q.shape[0]), float("nan"), dtype=torch.float64)
    lse_t = torch.zeros_like(lse)
    for b in range(len(cu_q) - 1):
        rq, rk = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        if nq == 0:
            continue
        keep = torch.ones(nq, nk, dtype=torch.bool)
        if causal:
            keep = keep.tril(nk - nq)
            if window:
                keep = keep.triu(nk - nq - window + 1)
        for h in range(heads):
            c = slice(h * hd, (h + 1) * hd)
            ck = slice(h // G * hd, (h // G + 1) * hd)
            a, kk, vv, dd = q[rq, c], k[rk, ck], v[rk, ck], do[rq, c]
            s = torch.where(keep, scale * (a @ kk.T), torch.tensor(-math.inf).double())
            if nk == 0:
                lse[h, rq] = -math.inf
                continue
            lse[h, rq] = torch.logsumexp(s, 1)
            p = torch.nan_to_num(torch.softmax(s, 1), nan=0.0)
            sabs = torch.where(keep, scale * (a.abs() @ kk.abs().T), torch.zeros(()).double())
            se = ((contraction_error(hd) + 4 * E) * sabs).amax(1, keepdim=True)  # one bound per row
            pe = 2 * se + 64 * E * (1 + sabs.amax(1, keepdim=True))
            lse_t[h, rq] = (se + 32 * E * (1 + sabs.amax(1, keepdim=True))).squeeze(1) + \
                contraction_error(nk)
            ov = p @ vv
            o[rq, c] = ov
            o_e = (pe + U + contraction_error(nk)) * (p @ vv.abs())
            o_t[rq, c] = U * ov.abs() + (1 + U) * o_e
            dv[rk, ck] += p.T @ dd
            pd = p.T @ dd.abs()
            dv_t[rk, ck] += (p * pe).T @ dd.abs() + (U + contraction_error(nq * G)) * pd
            dp = dd @ vv.T
            delta = (dd * ov).sum(1, keepdim=True)
            # delta is formed from the rounded O, dP in fp32
            de = (dd.abs() * o_t[rq, c]).sum(1, keepdim=True) + \
                contraction_error(hd) * (dd.abs() * ov.abs()).sum(1, keepdim=True)
            dpe = contraction_error(hd) * (dd.abs() @ vv.abs().T)
            ds = p * (dp - delta)
            ds_e = p * (dpe + de) + (pe + U + 4 * E) * ds.abs() + 2 * E * p * (dp.abs() + delta.abs())
            dq[rq, c] = scale * (ds @ kk)
            dq_t[rq, c] = U * dq[rq, c].abs() + (1 + U) * scale * (
                ds_e @ kk.abs() + contraction_error(nk) * (ds.abs() @ kk.abs()))
            dk[rk, ck] += scale * (ds.T @ a)
            dk_t[rk, ck] += scale * (ds_e.T @ a.abs() + contraction_error(nq * G) * (ds.abs().T @ a.abs()))
    dk_t = U * dk.abs() + (1 + U) * dk_t
    dv_t = U * dv.abs() + (1 + U) * dv_t
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv, "o_tol": o_t, "lse_tol": lse_t,
            "dq_tol": dq_t, "dk_tol": dk_t, "dv_tol": dv_t}


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
