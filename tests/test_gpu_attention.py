"""Attention on the GPU against the float64 form: every head layout, mask and
length where a tile, a block or a sequence ends, element by element."""
import math

import pytest
import torch

from lm_reference import attention, f64, within
from quantization_aware_tiny_b200 import qat

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


class Case:
    """Inputs of one call.  Rows behind the last sequence and columns beside the
    heads hold NaN in the inputs and a marker in the outputs."""

    def __init__(self, lq, lk=None, heads=4, kv_heads=2, hd=64, causal=True, window=0, scale=None,
                 pad=16, tail=3, packed=True, seed=0, peak=1.0):
        self.lq, self.lk = list(lq), list(lq if lk is None else lk)
        self.heads, self.kv_heads, self.hd = heads, kv_heads, hd
        self.causal, self.window, self.scale, self.packed = causal, window, scale, packed
        self.cu_q, self.cu_k = offsets(self.lq), offsets(self.lk)
        g = torch.Generator().manual_seed(seed + sum(self.lq) + 7 * sum(self.lk) + hd)
        tail = tail if packed else 0
        wq, wk, nq, nk = heads * hd, kv_heads * hd, self.cu_q[-1], self.cu_k[-1]

        def rows(n, width, std=1.0):
            x = torch.full((n + tail, width + pad), float("nan"), dtype=BF)
            x[:n, :width] = (torch.randn(n, width, generator=g) * std).to(BF)
            return x[:, :width], x.cuda()[:, :width]

        (self.q, self.Q), (self.k, self.K), (self.v, self.V), (self.do, self.dO) = (
            rows(nq, wq, peak), rows(nk, wk), rows(nk, wk), rows(nq, wq))
        self.nq, self.nk, self.tail, self.pad = nq, nk, tail, pad

    def out(self, n, width):
        return torch.full((n + self.tail, width + self.pad), 7.0, dtype=BF, device="cuda")

    def kw(self):
        d = dict(causal=self.causal, window=self.window, scale=self.scale)
        if self.packed:
            cu = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
            d.update(cu_q=cu(self.cu_q), cu_k=cu(self.cu_k), max_q=max(self.lq), max_k=max(self.lk))
        else:
            d.update(max_q=self.lq[0], max_k=self.lk[0])
        return d

    def forward(self, **more):
        wq = self.heads * self.hd
        o = self.out(self.nq, wq)
        lse = torch.full((self.heads, self.nq + self.tail), 7.0, device="cuda")
        qat.qat_attn_fwd(self.Q, self.K, self.V, o[:, :wq], lse, self.heads, self.kv_heads, self.hd,
                         **{**self.kw(), **more})
        return o, lse

    def reference(self):
        return attention(f64(self.q[:self.nq]), f64(self.k[:self.nk]), f64(self.v[:self.nk]),
                         f64(self.do[:self.nq]), self.heads, self.kv_heads, self.hd, self.cu_q, self.cu_k,
                         self.causal, self.window, self.scale or 1 / math.sqrt(self.hd))

    def compare(self, got, width, ref, tol, what):
        n = ref.shape[0]
        within(got[:n, :width], ref, tol, what)
        assert bool((got[n:] == 7).all()) and bool((got[:, width:] == 7).all()), what + ": rows beside"

    def check_forward(self):
        o, lse = self.forward()
        torch.cuda.synchronize()
        assert qat.device_error() == 0
        r = self.reference()
        self.compare(o, self.heads * self.hd, r["o"], r["o_tol"], "O")
        within(lse[:, :self.nq], r["lse"], r["lse_tol"], "lse")
        assert bool((lse[:, self.nq:] == 7).all())


MASKS = [dict(), dict(causal=False), dict(window=1), dict(window=37), dict(window=200)]
HEADS = [(4, 2, 64), (1, 1, 128), (2, 1, 80), (3, 3, 8), (4, 1, 24), (2, 2, 72), (4, 4, 120)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("causal", [True, False])
def test_fwd_head_layouts(heads, causal):
    h, kv, hd = heads
    Case([200, 1, 129], heads=h, kv_heads=kv, hd=hd, causal=causal).check_forward()


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 256, 257, 383, 600])
def test_fwd_lengths(n, mask):
    Case([n], heads=2, kv_heads=1, **mask).check_forward()


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("lens", [([64, 64], [300, 129]), ([300, 1, 5], [64, 1, 0]), ([130], [129]),
                                  ([1, 1, 1], [1, 200, 513]), ([0, 257, 0], [3, 257, 0])])
def test_fwd_queries_and_keys_of_other_lengths(lens, mask):
    """Fewer queries than keys, more queries than keys (rows that see nothing),
    single tokens, empty sequences."""
    Case(*lens, heads=2, kv_heads=2, hd=80, **mask).check_forward()


def test_fwd_equal_lengths_without_tables():
    Case([160] * 3, packed=False).check_forward()
    Case([64] * 3, [200] * 3, packed=False, hd=128).check_forward()


@pytest.mark.parametrize("peak", [0.0, 30.0])
def test_fwd_flat_and_peaked_rows(peak):
    """Equal scores, and scores whose maximum moves by hundreds from block to block."""
    Case([700], heads=1, kv_heads=1, peak=peak).check_forward()


def test_fwd_scale():
    Case([150], scale=0.7).check_forward()


def test_fwd_no_keys_at_all():
    Case([5, 3], [0, 0]).check_forward()


def test_fwd_nan_of_another_sequence_stays_there():
    """The second sequence is NaN throughout: the others are as if it were not there."""
    c = Case([100, 70, 90], tail=0)
    want = c.forward()
    for t in (c.Q, c.K, c.V):
        t[100:170] = float("nan")
    got = c.forward()
    torch.cuda.synchronize()
    keep = torch.ones(260, dtype=torch.bool, device="cuda")
    keep[100:170] = False
    assert torch.equal(want[0][keep], got[0][keep]) and torch.equal(want[1][:, keep], got[1][:, keep])
    assert bool(torch.isnan(got[0][100:170, :256]).all())


def test_fwd_offsets_past_32_bits():
    """Row offsets beyond 2^31 elements."""
    n, ld = 300, 1 << 23
    big = torch.empty(n, ld, dtype=BF, device="cuda")
    c = Case([n], heads=1, kv_heads=1, pad=0, tail=0)
    big[:, :64], big[:, 64:128], big[:, 128:192] = c.Q, c.K, c.V
    want, lse = c.forward()
    lse2 = torch.empty_like(lse)
    qat.qat_attn_fwd(big[:, :64], big[:, 64:128], big[:, 128:192], big[:, 192:256], lse2, 1, 1, 64, max_q=n)
    torch.cuda.synchronize()
    assert torch.equal(big[:, 192:256], want) and torch.equal(lse, lse2)
