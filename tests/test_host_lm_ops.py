"""Host-side argument checks of the language-model operators' C entry points:
every refusal happens before a launch, so none of this needs a GPU."""
import ctypes
import math

import pytest
import torch

from quantization_aware_tiny_b200 import qat

A16 = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10002)
BIG = 1 << 40


def L():
    return qat.lib()


def operand(N, K, ptr=0x10000):
    return ctypes.byref(qat._QWeight(ptr, None, None, N, K, 8))


def ce_fwd(W=None, qw=None, V=64, d=64, bits=8, Z=A16, ldz=0, T=8, targets=A16, loss=A16, lse=A16,
           mean=None, ws=A16, wsb=BIG):
    return L().qat_ce_fwd(W, qw, V, d, bits, Z, ldz, T, targets, loss, lse, mean, ws, wsb, None)


def ce_bwd(W=None, qw=None, V=64, d=64, bits=8, Z=A16, ldz=0, T=8, targets=A16, lse=A16, dloss=None,
           gscale=None, dZ=A16, dW=None, acc=0, ws=A16, wsb=BIG):
    return L().qat_ce_bwd(W, qw, V, d, bits, Z, ldz, T, targets, lse, dloss, gscale, dZ, dW, acc, ws,
                          wsb, None)


@pytest.mark.parametrize("call", [ce_fwd, ce_bwd])
def test_ce_refusals(call):
    before = qat.launch_count()
    q = operand(64, 64)
    for rc, kw in ((qat.QAT_ERR_ARG, dict(Z=None)), (qat.QAT_ERR_ARG, dict(targets=None)),
                   (qat.QAT_ERR_ARG, dict(lse=None)), (qat.QAT_ERR_ARG, dict(bits=7)),
                   (qat.QAT_ERR_ARG, dict(T=-1)), (qat.QAT_ERR_ARG, dict(V=0)),
                   (qat.QAT_ERR_ARG, dict(W=A16)), (qat.QAT_ERR_ARG, dict(qw=None)),
                   (qat.QAT_ERR_ARG, dict(qw=operand(64, 72))), (qat.QAT_ERR_SHAPE, dict(d=68)),
                   (qat.QAT_ERR_SHAPE, dict(V=(1 << 20) + 1)), (qat.QAT_ERR_SHAPE, dict(ldz=56)),
                   (qat.QAT_ERR_SHAPE, dict(ldz=68)), (qat.QAT_ERR_SHAPE, dict(T=1 << 31)),
                   (qat.QAT_ERR_ALIGN, dict(Z=ODD)), (qat.QAT_ERR_ALIGN, dict(targets=ODD)),
                   (qat.QAT_ERR_ALIGN, dict(lse=ODD)), (qat.QAT_ERR_ALIGN, dict(ws=ODD)),
                   (qat.QAT_ERR_ALIGN, dict(qw=operand(64, 64, 0x10008))),
                   (qat.QAT_ERR_WORKSPACE, dict(ws=None, wsb=0)),
                   (qat.QAT_ERR_WORKSPACE, dict(wsb=256)),
                   (qat.QAT_ERR_WORKSPACE, dict(W=A16, qw=None, wsb=300))):
        assert call(**{**dict(qw=q), **kw}) == rc, kw
    assert qat.launch_count() == before


def test_ce_bwd_without_outputs_does_nothing():
    assert ce_bwd(qw=operand(64, 64), dZ=None) == qat.QAT_OK
    for kw in (dict(dZ=ODD), dict(dW=ODD), dict(dloss=ODD), dict(gscale=ODD)):
        assert ce_bwd(**{**dict(qw=operand(64, 64)), **kw}) == qat.QAT_ERR_ALIGN


def test_ce_workspace_sizes():
    """The backward's size serves the forward; both grow with raw weights, and
    the pieces stay under about 1 GiB whatever the batch."""
    for V, d, T in ((8192, 512, 65536), (50257, 640, 4099), (1, 8, 1), (1 << 20, 64, 1000)):
        f = qat.workspace_size(qat.QAT_OP_CE_FWD, V, d, T, False)
        b = qat.workspace_size(qat.QAT_OP_CE_BWD, V, d, T, False)
        assert 0 < f <= b
        assert qat.workspace_size(qat.QAT_OP_CE_BWD, V, d, T, True) >= b + V * d * 2
        assert b <= max(f, (1 << 30) + 256 * 4 * (V + 8) + (1 << 20))
    assert qat.workspace_size(qat.QAT_OP_CE_FWD, 64, 64, 0, False) == 0


def test_ce_workspace_of_the_longest_batch_serves_shorter_ones():
    for V, d in ((64, 64), (1024, 512), (50257, 640)):
        sizes = [qat.workspace_size(qat.QAT_OP_CE_FWD, V, d, T, False) for T in range(1, 2100)]
        assert sizes == sorted(sizes)


# ------------------------------------------------------------------- rotary

def rope(X=A16, ldx=0, Y=ctypes.c_void_p(0x20000), ldy=0, dtype=1, T=4, heads=2, hd=64, rot=64, freqs=A16,
         scale=1.0, pos=None, seq=0):
    return L().qat_rope(X, ldx, Y, ldy, dtype, T, heads, hd, rot, freqs, scale, pos, seq, 0, 0, None)


def test_rope_refusals():
    before = qat.launch_count()
    for rc, kw in ((qat.QAT_ERR_ARG, dict(X=None)), (qat.QAT_ERR_ARG, dict(Y=None)),
                   (qat.QAT_ERR_ARG, dict(freqs=None)), (qat.QAT_ERR_ARG, dict(T=-1)),
                   (qat.QAT_ERR_ARG, dict(heads=0)), (qat.QAT_ERR_ARG, dict(dtype=2)),
                   (qat.QAT_ERR_ARG, dict(seq=-1)), (qat.QAT_ERR_SHAPE, dict(rot=63)),
                   (qat.QAT_ERR_SHAPE, dict(rot=66)), (qat.QAT_ERR_SHAPE, dict(rot=0)),
                   (qat.QAT_ERR_SHAPE, dict(hd=60, rot=60)), (qat.QAT_ERR_SHAPE, dict(ldx=120)),
                   (qat.QAT_ERR_SHAPE, dict(ldy=132)),
                   (qat.QAT_ERR_SHAPE, dict(hd=2048, rot=1026)), (qat.QAT_ERR_ALIGN, dict(X=ODD)),
                   (qat.QAT_ERR_ALIGN, dict(Y=ODD)), (qat.QAT_ERR_ALIGN, dict(freqs=ODD)),
                   (qat.QAT_ERR_ALIGN, dict(pos=ODD)),
                   (qat.QAT_ERR_ARG, dict(Y=A16, ldx=128, ldy=136))):
        assert rope(**kw) == rc, kw
    assert rope(T=0, X=None, Y=None) == qat.QAT_OK
    assert qat.launch_count() == before


def test_rope_freqs_are_the_formulas():
    """Plain and linear term by term; NTK keeps the first pair and slows the last by the
    factor; YaRN keeps fast pairs, divides slow ones, and 1 is its own scaling."""
    n = 32
    plain, m = qat.rope_freqs(2 * n, 10000.0, device="cpu")
    assert m == 1.0
    for i in range(n):
        assert float(plain[i]) == pytest.approx(10000.0 ** (-i / n) / (2 * math.pi), rel=1e-15)
    lin, _ = qat.rope_freqs(2 * n, 10000.0, "linear", 4.0, device="cpu")
    assert torch.equal(lin, plain / 4)
    ntk, _ = qat.rope_freqs(2 * n, 10000.0, "ntk", 4.0, device="cpu")
    assert float(ntk[0]) == float(plain[0])
    assert float(ntk[-1]) == pytest.approx(float(plain[-1]) / 4, rel=1e-12)
    yarn, m = qat.rope_freqs(2 * n, 10000.0, "yarn", 16.0, trained_len=1024, device="cpu")
    assert m == pytest.approx(0.1 * math.log(16.0) + 1.0)
    turns = plain * 1024
    assert torch.equal(yarn[turns > 64], plain[turns > 64])
    assert torch.allclose(yarn[turns < 0.5], plain[turns < 0.5] / 16, rtol=1e-15)
    assert bool((yarn <= plain).all()) and bool((yarn >= plain / 16 * (1 - 1e-15)).all())
    same, m = qat.rope_freqs(2 * n, 10000.0, "yarn", 1.0, trained_len=1024, device="cpu")
    assert m == 1.0 and torch.allclose(same, plain, rtol=1e-15)
    for bad in (dict(rotary=3), dict(rotary=0), dict(rotary=8, scaling="other"), dict(rotary=8, base=1.0),
                dict(rotary=8, scaling="linear", factor=0.5), dict(rotary=8, scaling="yarn", factor=2.0),
                dict(rotary=8, scaling="yarn", factor=2.0, trained_len=64, beta_fast=1.0, beta_slow=1.0),
                dict(rotary=8, base=float("nan")), dict(rotary=1026)):
        with pytest.raises(qat.QatError):
            qat.rope_freqs(device="cpu", **bad)


# ---------------------------------------------------------------- attention

def attn(Q=A16, K=A16, V=A16, O=A16, lse=A16, **kw):
    d = dict(Tq=64, Tk=64, cu_q=None, cu_k=None, batch=1, max_q=64, max_k=64, heads=4, kv_heads=2,
             head_dim=64, causal=1, window=0, scale=0.0, reserved=0, ldq=0, ldk=0, ldv=0, ldo=0)
    grad = {k: kw.pop(k) for k in ("lddo", "lddq", "lddk", "lddv", "dO", "dQ", "dK", "dV", "ws", "wsb") if k in kw}
    a = ctypes.byref(qat._Attn(**{**d, **kw}))
    if not grad:
        return L().qat_attn_fwd(a, Q, K, V, O, lse, None)
    g = lambda k: grad.get(k, 0 if k.startswith("ld") else A16)
    return L().qat_attn_bwd(a, g("dO"), g("lddo"), Q, K, V, O, lse, g("dQ"), g("lddq"), g("dK"), g("lddk"),
                            g("dV"), g("lddv"), g("ws"), grad.get("wsb", BIG), None)


def test_attention_refusals():
    before = qat.launch_count()
    nan, inf = float("nan"), float("inf")
    cases = [(qat.QAT_ERR_ARG, dict(Q=None)), (qat.QAT_ERR_ARG, dict(K=None)), (qat.QAT_ERR_ARG, dict(V=None)),
             (qat.QAT_ERR_ARG, dict(O=None)), (qat.QAT_ERR_ARG, dict(lse=None)), (qat.QAT_ERR_ARG, dict(Tq=-1)),
             (qat.QAT_ERR_ARG, dict(heads=0)), (qat.QAT_ERR_ARG, dict(kv_heads=3)),
             (qat.QAT_ERR_ARG, dict(kv_heads=0)), (qat.QAT_ERR_ARG, dict(window=-1)),
             (qat.QAT_ERR_ARG, dict(window=3, causal=0)), (qat.QAT_ERR_ARG, dict(scale=nan)),
             (qat.QAT_ERR_ARG, dict(scale=inf)), (qat.QAT_ERR_ARG, dict(scale=-1.0)),
             (qat.QAT_ERR_ARG, dict(Tq=65)), (qat.QAT_ERR_ARG, dict(Tk=32)), (qat.QAT_ERR_ARG, dict(batch=-1)),
             (qat.QAT_ERR_SHAPE, dict(head_dim=60)), (qat.QAT_ERR_SHAPE, dict(head_dim=136)),
             (qat.QAT_ERR_SHAPE, dict(head_dim=0)), (qat.QAT_ERR_SHAPE, dict(ldq=248)),
             (qat.QAT_ERR_SHAPE, dict(ldk=132)), (qat.QAT_ERR_SHAPE, dict(ldo=260)),
             (qat.QAT_ERR_SHAPE, dict(ldv=1 << 40)),
             (qat.QAT_ERR_SHAPE, dict(Tq=(1 << 31) - 1, batch=1, max_q=(1 << 31) - 1)),
             (qat.QAT_ERR_ALIGN, dict(Q=ODD)), (qat.QAT_ERR_ALIGN, dict(lse=ODD)),
             (qat.QAT_ERR_ALIGN, dict(cu_q=0x10002))]
    for rc, kw in cases:
        assert attn(**kw) == rc, kw
        assert attn(dO=A16, **kw) == rc, kw
    for rc, kw in ((qat.QAT_ERR_ARG, dict(dO=None)), (qat.QAT_ERR_ARG, dict(dQ=None)),
                   (qat.QAT_ERR_ARG, dict(dK=None)), (qat.QAT_ERR_ARG, dict(dV=None)),
                   (qat.QAT_ERR_SHAPE, dict(lddo=100)), (qat.QAT_ERR_SHAPE, dict(lddq=260)),
                   (qat.QAT_ERR_SHAPE, dict(lddk=64)), (qat.QAT_ERR_ALIGN, dict(dV=ODD)),
                   (qat.QAT_ERR_ALIGN, dict(ws=ODD)), (qat.QAT_ERR_WORKSPACE, dict(ws=None)),
                   (qat.QAT_ERR_WORKSPACE, dict(wsb=4 * 64 * 4 - 1))):
        assert attn(**kw) == rc, kw
    # nothing to do: no sequences, no rows
    assert attn(batch=0, Tq=0, Tk=0) == qat.QAT_OK and attn(dO=A16, batch=0, Tq=0, Tk=0) == qat.QAT_OK
    assert attn(batch=3, Tq=0, max_q=0, Tk=192) == qat.QAT_OK
    assert attn(dO=A16, batch=3, Tq=0, max_q=0, Tk=0, max_k=0) == qat.QAT_OK
    assert qat.launch_count() == before


# --------------------------------------------------- outputs in inputs' places

def test_outputs_in_the_place_of_inputs_are_refused():
    P = [ctypes.c_void_p(0x100000 * i) for i in range(1, 10)]
    Q, K, V, O, dO, dQ, dK, dV, lse = P
    before = qat.launch_count()
    for at in (Q, K, V):
        assert attn(Q=Q, K=K, V=V, O=at, lse=lse) == qat.QAT_ERR_ARG
    base = dict(Q=Q, K=K, V=V, O=O, lse=lse, dO=dO, dQ=dQ, dK=dK, dV=dV)
    for name in ("dQ", "dK", "dV"):
        for at in (Q, K, V, O, dO) + tuple(base[n] for n in ("dQ", "dK", "dV") if n != name):
            assert attn(**{**base, name: at}) == qat.QAT_ERR_ARG, name
    for dW in (None, O):
        assert ce_bwd(qw=operand(64, 64), Z=Q, dZ=Q, dW=dW) == qat.QAT_ERR_ARG
    assert qat.launch_count() == before


# ------------------------------------------------------------------ binding

def test_rows_that_share_memory_are_refused():
    """A broadcast row (the gradient of a sum) has stride 0, which the C side takes for
    contiguous rows: it would read memory behind the tensor."""
    row = torch.zeros(1, 64)
    for t in (row.expand(8, 64), torch.zeros(100).as_strided((3, 64), (8, 1))):
        with pytest.raises(qat.QatError) as e:
            qat._rows("call", t, 64)
        assert e.value.code == qat.QAT_ERR_ARG
    wide = torch.zeros(8, 200)
    assert qat._rows("call", wide[:, 8:72], 64) == 200
    # the stride of a single row, or of none, says nothing
    assert qat._rows("call", row.expand(1, 64), 64) == qat._rows("call", torch.zeros(1, 203)[:, :64], 64) == 64
    assert qat._rows("call", wide[:0, :64], 64) == 64


def test_attention_arguments_that_32_bits_do_not_hold(monkeypatch):
    """What the C side would wrap to another value, take for its default, or cut every
    sequence to: refused before a tensor is looked at."""
    monkeypatch.setattr(qat, "_need", lambda *a: None)
    rows = lambda w: torch.zeros(64, w, dtype=torch.bfloat16)
    q, k, lse = rows(128), rows(64), torch.zeros(2, 64)
    cu = torch.tensor([0, 64], dtype=torch.int32)

    def descriptor(heads=2, kv=1, hd=64, window=0, scale=None, cu_q=cu, cu_k=None, max_q=64, max_k=None):
        return qat._attn("call", q, k, k, q, lse, heads, kv, hd, True, window, scale, cu_q, cu_k, max_q, max_k)

    a = descriptor(window=(1 << 31) - 1, scale=2.0 ** -126)
    assert (a.batch, a.max_q, a.max_k, a.window, a.scale) == (1, 64, 64, (1 << 31) - 1, 2.0 ** -126)
    a = descriptor(cu_q=None)
    assert (a.batch, a.max_k, a.cu_k, a.scale) == (1, 64, None, 0.0)
    for kw in (dict(window=1 << 32), dict(window=-1), dict(scale=0.0), dict(scale=1e-46), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(max_q=None), dict(max_q=1 << 32),
               dict(cu_k=cu), dict(cu_q=None, max_q=None), dict(cu_q=None, max_q=None, max_k=64)):
        with pytest.raises(qat.QatError) as e:
            descriptor(**kw)
        assert e.value.code == qat.QAT_ERR_ARG, kw
