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


# ------------------------------------------------ memory that arguments share

# More query blocks than a grid holds: such a call is refused after its arguments have been
# looked at and before anything is launched, so made-up addresses are safe everywhere.
TOO_LONG = (1 << 31) - 1


def runs(at, rows, ld, cols):
    """Byte ranges of a bf16 row tensor."""
    return [(at + 2 * ld * i, at + 2 * (ld * i + cols)) for i in range(rows)]


def meet(a, b):
    return any(x0 < y1 and y0 < x1 for x0, x1 in a for y0, y1 in b)


def test_overlap_is_found_exactly():
    """Two row tensors of any starts, strides and lengths, against their byte ranges."""
    import random
    rng = random.Random(5)
    base, before, seen = 0x4000000000, qat.launch_count(), [0, 0]
    P = [at(0x10000000 * i) for i in range(1, 9)]
    for n in range(4000):
        H, KH, hd = rng.choice([(1, 1, 8), (2, 1, 8), (3, 1, 16)])
        wq, wk = H * hd, KH * hd
        Tq, Tk = rng.randint(1, 9), rng.randint(1, 9)
        ldq, ldk = wq + 8 * rng.randint(0, 8), wk + 8 * rng.randint(0, 8)
        if n % 3 == 0:
            ldk = ldq if wk <= ldq else ldk
        o, k = base + 16 * rng.randint(0, 90), base + 16 * rng.randint(0, 90)
        shared = meet(runs(o, Tq, ldq, wq), runs(k, Tk, ldk, wk))
        seen[shared] += 1
        want = qat.QAT_ERR_ARG if shared else None
        kw = dict(Tq=Tq, Tk=Tk, heads=H, kv_heads=KH, head_dim=hd, batch=1, max_q=TOO_LONG, max_k=TOO_LONG,
                  cu_q=0x5000, cu_k=0x6000)
        fwd = attn(Q=P[0], K=at(k), V=P[1], O=at(o), lse=P[2], ldk=ldk, ldo=ldq, **kw)
        bwd = attn(Q=P[0], K=P[1], V=P[2], O=P[3], lse=P[4], dO=P[5], dQ=at(o), dK=at(k), dV=P[6], lddq=ldq, lddk=ldk,
                   ws=P[7], **kw)
        inp = attn(Q=P[0], K=P[1], V=at(k), O=P[3], lse=P[4], dO=P[5], dQ=at(o), dK=P[2], dV=P[6], lddq=ldq, ldv=ldk,
                   ws=P[7], **kw)
        for rc in (fwd, bwd, inp):
            assert rc != qat.QAT_OK and (rc == qat.QAT_ERR_ARG) == shared, (n, rc, shared)
    assert min(seen) > 500 and qat.launch_count() == before


def test_overlapping_views_are_refused():
    """Not only equal addresses: a view from another offset, statistics in a row tensor's
    memory, the workspace in an argument's."""
    before = qat.launch_count()
    T, V, d = 8, 64, 64
    A = {n: 0x10000000 * i for i, n in enumerate(("Z", "targets", "loss", "lse", "mean", "ws", "dZ", "dW", "dloss",
                                                   "gscale", "op"), 1)}
    sizes = dict(Z=T * d * 2, targets=T * 8, loss=T * 4, lse=T * 4, mean=8, dZ=T * d * 2, dW=V * d * 4, dloss=T * 4,
                 gscale=4, op=V * d * 2)

    def ce(call, names, **moved):
        a = {**A, **moved}
        return call(qw=operand(V, d, a["op"]), V=V, d=d, T=T, **{n: at(a[n]) for n in names})

    fwd, bwd = ("Z", "targets", "loss", "lse", "mean", "ws"), ("Z", "targets", "lse", "dloss", "gscale", "dZ", "dW", "ws")
    for call, names, outs in ((ce_fwd, fwd, ("loss", "lse", "mean")), (ce_bwd, bwd, ("dZ", "dW"))):
        for out in outs:
            for other in names + ("op",):
                if other == out:
                    continue
                end = 16 if other == "ws" else sizes[other] // 16 * 16 - 16
                assert ce(call, names, **{out: A[other] + max(end, 0)}) == qat.QAT_ERR_ARG, (out, other)
                if other in sizes and sizes[out] > 16:
                    back = (sizes[out] - 1) // 16 * 16
                    assert ce(call, names, **{out: A[other] - back}) == qat.QAT_ERR_ARG, (out, other)
    assert rope(X=at(0x10000), Y=at(0x10000 + 16), T=4) == qat.QAT_ERR_ARG
    assert rope(X=at(0x10000), Y=at(0x10000 + 3 * 256), T=4) == qat.QAT_ERR_ARG
    assert rope(X=at(0x10000), Y=at(0x30000), freqs=at(0x30000 + 512), T=4) == qat.QAT_ERR_ARG
    assert rope(X=at(0x10000), Y=at(0x30000), pos=at(0x30000 - 24), T=4) == qat.QAT_ERR_ARG
    q = dict(Q=at(0x100000), K=at(0x200000), V=at(0x300000), O=at(0x400000), lse=at(0x500000))
    assert attn(**{**q, "lse": at(0x400000 + 64)}) == qat.QAT_ERR_ARG
    assert attn(**q, dO=at(0x600000), dQ=at(0x700000), dK=at(0x800000), dV=at(0x900000),
                ws=at(0x500000 + 512)) == qat.QAT_ERR_ARG
    assert attn(**{**q, "cu_q": 0x400000 + 4}) == qat.QAT_ERR_ARG
    assert qat.launch_count() == before


# ------------------------------------------------------------------ binding

def descriptor(monkeypatch, Tq, Tk, **kw):
    monkeypatch.setattr(qat, "_need", lambda *a: None)
    rows = lambda n, w: torch.zeros(n, w, dtype=torch.bfloat16)
    q, k = rows(Tq, 128), rows(Tk, 64)
    d = dict(cu_q=None, cu_k=None, max_q=None, max_k=None)
    return qat._attn("call", q, k, k, q, torch.zeros(2, Tq), 2, 1, 64, True, 0, None, **{**d, **kw})


def test_no_keys_is_not_keys_as_queries(monkeypatch):
    """max_k = 0 says that no sequence has a key; only max_k left out says that the keys
    lie as the queries do."""
    cu = torch.tensor([0, 3, 7], dtype=torch.int32)
    a = descriptor(monkeypatch, 7, 0, cu_q=cu, max_q=4, max_k=0)
    assert (a.batch, a.Tq, a.Tk, a.max_q, a.max_k, a.cu_k) == (2, 7, 0, 4, 0, None)
    a = descriptor(monkeypatch, 8, 0, max_q=4, max_k=0)
    assert (a.batch, a.max_k, a.cu_k) == (2, 0, None)
    a = descriptor(monkeypatch, 7, 7, cu_q=cu, max_q=4)
    assert (a.batch, a.max_k) == (2, 4) and a.cu_k == a.cu_q


def test_workspaces_that_hold_less_than_they_count_are_refused(monkeypatch):
    """The C side takes an address and a size: broadcast or gapped workspaces, and those of
    another device, never reach it."""
    place = [0]  # of the current device; host tensors are on none (-1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: place[0])
    whole = torch.zeros(64, dtype=torch.uint8)
    for ws in (whole[:1].expand(1 << 20), whole[::2], whole):
        with pytest.raises(qat.QatError) as e:
            qat._scratch("call", ws)
        assert e.value.code == qat.QAT_ERR_ARG
    place[0] = -1
    assert qat._scratch("call", whole[16:]) == (whole.data_ptr() + 16, 48)
    assert qat._scratch("call", None) == (None, 0)
    for ws in (whole[:1].expand(1 << 20), whole[::2]):
        with pytest.raises(qat.QatError):
            qat._scratch("call", ws)


def test_rope_freqs_of_more_dims_than_32_bits_hold():
    """Refused before the table is made (of 2^31 pairs) and not taken as 8 dims."""
    for rotary in ((1 << 32) + 8, 1 << 40, qat.QAT_ROPE_MAX_DIMS + 2):
        with pytest.raises(qat.QatError) as e:
            qat.rope_freqs(rotary, device="cpu")
        assert e.value.code == qat.QAT_ERR_SHAPE


def test_walks_that_would_outlast_the_bounded_waits_are_refused():
    """More than 2^26 keys under more than 128 queries: one tile of a piece would wait for the
    other's whole walk."""
    P = [at(0x10000000 * i) for i in range(1, 6)]
    keys = (1 << 26) + 1
    long = dict(Q=P[0], K=at(0x1000000000), V=at(0x9000000000), O=P[3], lse=P[4], heads=1, kv_heads=1, head_dim=8,
                max_q=129, Tq=129, max_k=keys, Tk=keys)
    before = qat.launch_count()
    assert attn(**long) == qat.QAT_ERR_SHAPE
    assert attn(**{**long, "cu_k": 0x5000, "max_k": TOO_LONG}) == qat.QAT_ERR_SHAPE
    assert qat.launch_count() == before
