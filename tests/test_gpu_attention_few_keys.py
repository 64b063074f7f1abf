"""Attention gradients of queries that see few keys, element by element: dS there is a
difference of near numbers, so delta = rowsum(dO * O) has to be better than the bf16 O."""
import math

import pytest
import torch

from lm_reference import E, U, contraction_error
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


def reference(c):
    """Float64 dQ and dK with bounds in which delta is good to the scores' own accuracy.

    With P off by the relative amount pe and dP by dpe, sum(P dP) is off by sum(P dpe) and,
    since sum(P (dP - delta)) = 0, by no more than pe times sum(P |dP - delta|) and pe
    times what the first guess of delta (from the rounded O and P: at most 4 U of
    sum |dO| |P V|) was off; then fp32 sums.  dS and the results are rounded once more."""
    H, G, hd, scale = c.heads, c.heads // c.kv_heads, c.hd, c.scale or 1 / math.sqrt(c.hd)
    q, k, v, do = (t.double() for t in (c.q[:c.nq], c.k[:c.nk], c.v[:c.nk], c.do[:c.nq]))
    dq, dk = torch.zeros_like(q), torch.zeros_like(k)
    dq_t, dk_t = torch.zeros_like(q), torch.zeros_like(k)
    for b in range(len(c.lq)):
        rq, rk = slice(c.cu_q[b], c.cu_q[b + 1]), slice(c.cu_k[b], c.cu_k[b + 1])
        nq, nk = c.lq[b], c.lk[b]
        if nq == 0 or nk == 0:
            continue
        keep = torch.ones(nq, nk, dtype=torch.bool)
        if c.causal:
            keep = keep.tril(nk - nq)
            if c.window:
                keep = keep.triu(nk - nq - c.window + 1)
        for h in range(H):
            cq, ck = slice(h * hd, (h + 1) * hd), slice(h // G * hd, (h // G + 1) * hd)
            a, kk, vv, dd = q[rq, cq], k[rk, ck], v[rk, ck], do[rq, cq]
            s = torch.where(keep, scale * (a @ kk.T), torch.tensor(-math.inf).double())
            p = torch.nan_to_num(torch.softmax(s, 1), nan=0.0)
            sabs = torch.where(keep, scale * (a.abs() @ kk.abs().T), torch.zeros(()).double())
            top = sabs.amax(1, keepdim=True)
            pe = 2 * (contraction_error(hd) + 4 * E) * top + 64 * E * (1 + top)
            dp = dd @ vv.T
            delta = (p * dp).sum(1, keepdim=True)
            ds = p * (dp - delta)
            dpe = contraction_error(hd) * (dd.abs() @ vv.abs().T)
            guess = 4 * U * (dd.abs() * (p @ vv.abs())).sum(1, keepdim=True)
            de = (p * dpe).sum(1, keepdim=True) + (pe + contraction_error(nk) + 64 * E) * (
                ds.abs().sum(1, keepdim=True) + guess) + 4 * E * (delta.abs() + guess)
            ds_e = p * (dpe + de) + (pe + U + 4 * E) * ds.abs() + 2 * E * p * (dp.abs() + delta.abs())
            ds_e = torch.where(keep.sum(1, keepdim=True) == 1, torch.zeros(()).double(), ds_e)
            dq[rq, cq] = scale * (ds @ kk)
            dq_t[rq, cq] = U * dq[rq, cq].abs() + (1 + U) * scale * (
                ds_e @ kk.abs() + contraction_error(nk) * (ds.abs() @ kk.abs()))
            dk[rk, ck] += scale * (ds.T @ a)
            dk_t[rk, ck] += scale * (ds_e.T @ a.abs() + contraction_error(nq * G) * (ds.abs().T @ a.abs()))
    return {"dq": (dq, dq_t), "dk": (dk, U * dk.abs() + (1 + U) * dk_t)}


def check(c, names=("dq", "dk")):
    from quantization_aware_tiny_b200 import qat
    o, lse = c.forward()
    grads = c.backward(o, lse)
    torch.cuda.synchronize()
    assert qat.device_error() == 0
    want = reference(c)
    for name, got in zip(("dq", "dk"), grads):
        if name in names:
            ref, tol = want[name]
            c.compare(got, ref.shape[1], ref, tol, name)


@pytest.mark.parametrize("peak", [1.0, 6.0])
@pytest.mark.parametrize("heads", [(2, 2, 40), (4, 1, 64), (2, 1, 128), (8, 2, 80)])
@pytest.mark.parametrize("causal", [False, True])
def test_few_keys(heads, causal, peak):
    """Two to sixteen keys under one to many queries, softmaxes of any shape."""
    H, KH, hd = heads
    check(Case([4, 330, 11, 1, 129, 200, 50], [2, 2, 5, 3, 16, 9, 2], heads=H, kv_heads=KH, hd=hd, causal=causal,
               peak=peak))


@pytest.mark.parametrize("peak", [1.0, 6.0])
@pytest.mark.parametrize("n", [2, 3, 16, 64, 127, 128])
def test_sequences_of_one_block(n, peak):
    check(Case([n, 1, n], heads=4, kv_heads=2, hd=72, peak=peak))
    check(Case([300, 40], [n, n], heads=4, kv_heads=2, hd=72, causal=False, peak=peak))


@pytest.mark.parametrize("peak", [1.0, 6.0])
@pytest.mark.parametrize("window", [2, 3, 8, 16])
@pytest.mark.parametrize("lens", [([300, 129, 5, 700], None), ([200, 300, 64], [500, 130, 700]), ([400, 140], [150, 129])])
def test_small_windows(lens, window, peak):
    """Tiles of queries whose few keys lie in more than one block."""
    for H, KH, hd in ((2, 1, 64), (3, 3, 104)):
        check(Case(*lens, heads=H, kv_heads=KH, hd=hd, window=window, peak=peak))


def test_key_gradients_of_long_rows():
    """dK of rows whose keys lie in many blocks: delta is mended before the second kernel."""
    for peak in (1.0, 6.0):
        check(Case([390, 257], heads=4, kv_heads=2, hd=64, peak=peak), names=("dk",))
        check(Case([200], [515], heads=2, kv_heads=2, hd=128, causal=False, peak=peak), names=("dk",))
