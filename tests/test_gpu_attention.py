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

    def backward(self, o, lse, **more):
        wq, wk = self.heads * self.hd, self.kv_heads * self.hd
        grads = self.out(self.nq, wq), self.out(self.nk, wk), self.out(self.nk, wk)
        ws = torch.full((qat.workspace_size(qat.QAT_OP_ATTN_BWD, self.heads, self.hd, self.Q.shape[0], False),),
                        255, dtype=torch.uint8, device="cuda")  # NaN
        qat.qat_attn_bwd(self.dO, self.Q, self.K, self.V, o[:, :wq], lse, grads[0][:, :wq],
                         grads[1][:, :wk], grads[2][:, :wk], self.heads, self.kv_heads, self.hd,
                         workspace=ws, **{**self.kw(), **more})
        return grads

    def check_backward(self):
        o, lse = self.forward()
        grads = self.backward(o, lse)
        torch.cuda.synchronize()
        assert qat.device_error() == 0
        r = self.reference()
        for name, g, heads in zip(("dq", "dk", "dv"), grads, (self.heads, self.kv_heads, self.kv_heads)):
            self.compare(g, heads * self.hd, r[name], r[name + "_tol"], name)

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
@pytest.mark.parametrize("n", [129, 256, 257, 383, 600])
def test_fwd_lengths_of_heads_that_share_nothing(n, mask):
    """As many key heads as query heads: both tiles are of one head."""
    Case([n, 40], heads=2, kv_heads=2, **mask).check_forward()


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("lens", [([64, 64], [300, 129]), ([300, 1, 5], [64, 1, 0]), ([130], [129]),
                                  ([1, 1, 1], [1, 200, 513]), ([0, 257, 0], [3, 257, 0])])
def test_fwd_queries_and_keys_of_other_lengths(lens, mask):
    """Fewer queries than keys, more queries than keys (rows that see nothing),
    single tokens, empty sequences."""
    Case(*lens, heads=2, kv_heads=2, hd=80, **mask).check_forward()


@pytest.mark.parametrize("heads", [(8, 1, 64), (8, 2, 80), (6, 2, 128), (3, 1, 32), (5, 5, 64), (12, 1, 16)])
@pytest.mark.parametrize("n", [1, 31, 33, 64, 65, 128])
def test_fwd_few_queries_over_many_keys(heads, n):
    """Heads of a group share a tile's rows, the two tiles share the keys: single
    tokens, rows off the tile, key counts of one block, an odd and an even number."""
    h, kv, hd = heads
    for window in (0, 150):
        Case([n, max(1, n // 2), n], [700, 100, 257], heads=h, kv_heads=kv, hd=hd, window=window).check_forward()


def test_fwd_more_pieces_than_the_gpu_holds():
    """Blocks take over pieces that have not started: thousands of them, empty ones among them."""
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 400, (300,), generator=g).tolist()
    Case(lens, heads=4, kv_heads=2, hd=16).check_forward()
    lq = torch.randint(0, 65, (700,), generator=g).tolist()
    lk = torch.randint(0, 300, (700,), generator=g).tolist()
    Case(lq, lk, heads=4, kv_heads=2, hd=16).check_forward()


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


# ------------------------------------------------------------------ backward

@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("causal", [True, False])
def test_bwd_head_layouts(heads, causal):
    h, kv, hd = heads
    Case([200, 1, 129], heads=h, kv_heads=kv, hd=hd, causal=causal).check_backward()


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 600])
def test_bwd_lengths(n, mask):
    Case([n], heads=2, kv_heads=1, **mask).check_backward()


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("lens", [([64, 64], [300, 129]), ([300, 1, 5], [64, 1, 0]), ([130], [129]),
                                  ([1, 1, 1], [1, 200, 513]), ([0, 257, 0], [3, 257, 0])])
def test_bwd_queries_and_keys_of_other_lengths(lens, mask):
    Case(*lens, heads=2, kv_heads=2, hd=80, **mask).check_backward()


def test_bwd_more_pieces_than_the_gpu_holds():
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 400, (300,), generator=g).tolist()
    Case(lens, heads=4, kv_heads=2, hd=16).check_backward()
    lq = torch.randint(0, 65, (700,), generator=g).tolist()
    lk = torch.randint(0, 300, (700,), generator=g).tolist()
    Case(lq, lk, heads=4, kv_heads=2, hd=104).check_backward()


def test_bwd_equal_lengths_without_tables():
    Case([160] * 3, packed=False).check_backward()
    Case([64] * 3, [200] * 3, packed=False, hd=128).check_backward()


@pytest.mark.parametrize("peak", [0.0, 5.0])
def test_bwd_flat_and_peaked_rows(peak):
    Case([700], heads=1, kv_heads=1, peak=peak).check_backward()


@pytest.mark.parametrize("kw", [dict(lq=[70, 3], window=1), dict(lq=[5, 300], lk=[1, 1], causal=False),
                                dict(lq=[5, 300], lk=[1, 1]), dict(lq=[1, 1, 1])])
def test_bwd_single_key_has_no_gradient(kw):
    """A softmax over one key is constant: dQ and dK are exactly zero."""
    c = Case(heads=2, kv_heads=1, hd=80, **kw)
    c.check_backward()
    o, lse = c.forward()
    dq, dk, dv = c.backward(o, lse)
    torch.cuda.synchronize()
    assert not dq[:c.nq, :160].any() and not dk[:c.nk, :80].any() and dv[:c.nk, :80].any()


def test_bwd_first_row_of_a_causal_sequence():
    """The row that sees key 0 only: its dQ is exactly zero, the next one's is not."""
    for lq, lk in (([200], [200]), ([300], [170])):
        c = Case(lq, lk, heads=2, kv_heads=2)
        o, lse = c.forward()
        dq = c.backward(o, lse)[0]
        torch.cuda.synchronize()
        first = lq[0] - lk[0]
        assert not dq[:first + 1, :128].any() and dq[first + 1, :128].any()


def test_bwd_scale():
    Case([150], scale=0.7).check_backward()


def test_bwd_no_keys_and_no_queries():
    """Without keys dQ is zero, without queries dK and dV are."""
    c = Case([5, 3], [0, 0])
    c.check_backward()
    Case([0, 0], [5, 3]).check_backward()


def test_bwd_nan_of_another_sequence_stays_there():
    c = Case([100, 70, 90], tail=0)
    o, lse = c.forward()
    want = c.backward(o, lse)
    for t in (c.Q, c.K, c.V, c.dO):
        t[100:170] = float("nan")
    o, lse = c.forward()
    got = c.backward(o, lse)
    torch.cuda.synchronize()
    keep = torch.ones(260, dtype=torch.bool, device="cuda")
    keep[100:170] = False
    for a, b in zip(want, got):
        assert torch.equal(a[keep], b[keep])


def test_bwd_gradients_into_one_projection_row():
    """dQ, dK, dV as the column ranges of one buffer, bit for bit."""
    c = Case([300], pad=0, tail=0)
    o, lse = c.forward()
    want = c.backward(o, lse)
    dqkv = torch.empty(300, 512, dtype=BF, device="cuda")
    ws = torch.empty(qat.workspace_size(qat.QAT_OP_ATTN_BWD, 4, 64, 300, False), dtype=torch.uint8, device="cuda")
    qat.qat_attn_bwd(c.dO, c.Q, c.K, c.V, o, lse, dqkv[:, :256], dqkv[:, 256:384], dqkv[:, 384:], 4, 2, 64,
                     workspace=ws, **c.kw())
    torch.cuda.synchronize()
    assert torch.equal(dqkv, torch.cat(want, 1))


def test_bwd_against_differences():
    """All three gradients along random directions against the difference quotient of
    the float64 form's sum(O * dO)."""
    c = Case([90, 33], heads=2, kv_heads=1, hd=24, pad=0, tail=0)
    o, lse = c.forward()
    grads = c.backward(o, lse)
    torch.cuda.synchronize()
    r, g = c.reference(), torch.Generator().manual_seed(5)
    base = [f64(t) for t in (c.q, c.k, c.v)]
    f = lambda x: float((attention(*x, f64(c.do), 2, 1, 24, c.cu_q, c.cu_k, True, 0, 24 ** -0.5)["o"] * f64(c.do)).sum())
    for at, (name, got) in enumerate(zip(("dq", "dk", "dv"), grads)):
        d, h = torch.randn(base[at].shape, generator=g).double(), 1e-5
        move = lambda e: [x + e * d if n == at else x for n, x in enumerate(base)]
        quotient = (f(move(h)) - f(move(-h))) / (2 * h)
        assert abs(float((f64(got) * d).sum()) - quotient) <= float((r[name + "_tol"] * d.abs()).sum()) + 1e-5


def test_same_bits_every_time_on_two_streams_and_in_a_graph():
    """Two calls at once on their own streams and workspaces, and a captured forward
    and backward replayed on new values while eager calls go on, give the eager bits."""
    c, c2 = Case([500, 77], seed=1, tail=0, pad=0), Case([500, 77], seed=2, tail=0, pad=0)

    def both(x):
        o, lse = x.forward()
        return (o, lse) + tuple(x.backward(o, lse))

    want, want2 = both(c), both(c2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a = both(c)
        with torch.cuda.stream(s2):
            b = both(c2)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, a))
        assert all(torch.equal(x, y) for x, y in zip(want2, b))
    kw = c.kw()
    c.kw = lambda: kw  # the tables are made once, outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s1), torch.cuda.graph(graph, stream=s1):
        got = both(c)
    keep = [t.clone() for t in (c.Q, c.K, c.V, c.dO)]
    for src, w in ((( c2.Q, c2.K, c2.V, c2.dO), want2), (keep, want)):
        for t, x in zip((c.Q, c.K, c.V, c.dO), src):
            t.copy_(x)
        graph.replay()
        both(c2)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(w, got))


def test_tables_that_do_not_fit_are_cut():
    """Offsets behind the tensors or before them, falling ones, and sequences longer
    than max_q / max_k: what is left of each is computed, the rest stays as it was."""
    c = Case([100, 60], tail=0, pad=0, heads=2, kv_heads=1)
    wide = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    want = Case([100, 60], tail=0, pad=0, heads=2, kv_heads=1)
    o, lse = want.forward()
    got, lse2 = c.forward(cu_q=wide([-7, 100, 999]), cu_k=wide([-7, 100, 999]))
    torch.cuda.synchronize()
    assert torch.equal(o, got) and torch.equal(lse, lse2)
    first = Case([64, 0, 60], [64, 0, 60], tail=0, pad=0, heads=2, kv_heads=1)
    for name in ("Q", "K", "V", "dO"):  # the first 64 rows of 100, and the second sequence
        src = getattr(c, name)
        setattr(first, name, torch.cat([src[:64], src[100:]]))
    fo, flse = first.forward()
    fg = first.backward(fo, flse)
    tab = dict(cu_q=wide([0, 100, 100, 160]), cu_k=wide([0, 100, 100, 160]), max_q=64, max_k=64)
    got, lse2 = c.forward(**tab)
    grads = c.backward(got, lse2, **tab)
    torch.cuda.synchronize()
    keep = torch.cat([torch.arange(64), torch.arange(100, 160)]).cuda()
    assert torch.equal(got[keep], fo) and bool((got[64:100] == 7).all())
    for a, b in zip(grads, fg):
        assert torch.equal(a[keep], b) and bool((a[64:100] == 7).all())
    falling, _ = c.forward(cu_q=wide([50, 20, 80]), cu_k=wide([50, 20, 80]))
    torch.cuda.synchronize()
    assert bool((falling[:20] == 7).all()) and bool((falling[80:] == 7).all()) and qat.device_error() == 0


def test_refusals():
    c = Case([64], tail=0, pad=0)
    o, lse = c.forward()
    ws = torch.empty(qat.workspace_size(qat.QAT_OP_ATTN_BWD, 4, 64, 64, False), dtype=torch.uint8, device="cuda")
    kw = c.kw()

    def bad(code, Q=c.Q, K=c.K, V=c.V, O=o, L=lse, heads=4, kv=2, hd=64, **k):
        with pytest.raises(qat.QatError) as e:
            qat.qat_attn_fwd(Q, K, V, O, L, heads, kv, hd, **{**kw, **k})
        assert e.value.code == code

    before = qat.launch_count()
    bad(qat.QAT_ERR_ARG, Q=c.Q.float())
    bad(qat.QAT_ERR_ARG, K=c.K.half())
    bad(qat.QAT_ERR_ARG, L=lse.double())
    bad(qat.QAT_ERR_ARG, L=lse[:3])
    bad(qat.QAT_ERR_ARG, O=o[:63])
    bad(qat.QAT_ERR_ARG, V=c.V[:63])
    bad(qat.QAT_ERR_ARG, Q=c.Q.cpu())
    bad(qat.QAT_ERR_ARG, heads=8)
    bad(qat.QAT_ERR_ARG, kv=3)
    bad(qat.QAT_ERR_ARG, cu_q=kw["cu_q"].long())
    bad(qat.QAT_ERR_ARG, cu_k=kw["cu_k"][:1])
    bad(qat.QAT_ERR_ARG, causal=False, window=4)
    bad(qat.QAT_ERR_ARG, cu_q=None, cu_k=None, max_q=60, max_k=60)
    bad(qat.QAT_ERR_SHAPE, heads=2, kv=1, hd=60)
    bad(qat.QAT_ERR_SHAPE, heads=1, kv=1, hd=136, K=torch.cat([c.K, c.K], 1), V=torch.cat([c.V, c.V], 1))
    with pytest.raises(qat.QatError) as e:
        qat.qat_attn_bwd(c.dO, c.Q, c.K, c.V, o, lse, o, c.K, c.V, 4, 2, 64, workspace=ws[:512], **kw)
    assert e.value.code == qat.QAT_ERR_WORKSPACE
    assert qat.launch_count() == before
