"""Refusals of the language-model operators that depend on more than one argument:
each comes before the first launch, so none of this needs a GPU."""
import ctypes

import pytest
import torch

from quantization_aware_tiny_b200 import qat
from test_host_lm_ops import attn, ce_bwd, ce_fwd, operand, rope

BIG = 1 << 40


def at(address):
    return ctypes.c_void_p(address)


def operand_bytes(V, d):
    up = lambda n: (n + 255) // 256 * 256
    return up(V * d * 2) + up(V * 4)


def test_ce_bwd_refuses_before_it_quantizes_the_head():
    """Raw fp32 words: the operand is made in the workspace, so a call that is refused
    must not have begun to."""
    V, d = 64, 64
    raw = dict(W=at(0x40000000), V=V, d=d, Z=at(0x10000000), dZ=at(0x20000000), ws=at(0x30000000))
    piece = 256 * V * 4 + 1024
    before = qat.launch_count()
    for T in (256, 1000):
        assert ce_bwd(T=T, wsb=operand_bytes(V, d) + piece - 1, **raw) == qat.QAT_ERR_WORKSPACE
        assert ce_bwd(T=T, wsb=operand_bytes(V, d), **raw) == qat.QAT_ERR_WORKSPACE
        assert ce_bwd(T=T, wsb=BIG, **{**raw, "dZ": raw["Z"]}) == qat.QAT_ERR_ARG
    for call in (ce_fwd, ce_bwd):
        rows = dict(W=raw["W"], V=V, d=d, Z=raw["Z"], ws=raw["ws"])
        assert call(ldz=(1 << 38) + 8, **rows) == qat.QAT_ERR_SHAPE
    assert qat.launch_count() == before
