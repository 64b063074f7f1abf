"""Host-side argument checks of the language-model operators' C entry points:
every refusal happens before a launch, so none of this needs a GPU."""
import ctypes

import pytest

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
