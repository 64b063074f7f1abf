"""Calls of the language-model operators that their documentation allows and that
lie off the ordinary path: values that are not finite, lengths given as zero,
far positions, memory that arguments share."""
import math

import pytest
import torch

from lm_reference import f64
from quantization_aware_tiny_b200 import qat

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def ce_loss(Z, targets, operand):
    """loss, lse and mean of one forward call."""
    T, (V, d) = Z.shape[0], operand.shape
    loss, lse, mean = (torch.full((n,), 7.0, device="cuda") for n in (T, T, 2))
    ws = torch.empty(qat.workspace_size(qat.QAT_OP_CE_FWD, V, d, T, False), dtype=torch.uint8, device="cuda")
    qat.qat_ce_fwd(Z.cuda(), targets.cuda(), loss, lse, 8, qw=qat.QWeight(operand.cuda(), None, None, 8),
                   mean=mean, workspace=ws)
    torch.cuda.synchronize()
    assert qat.device_error() == 0
    return loss, lse, mean


@pytest.mark.parametrize("T", [5, 1100])
@pytest.mark.parametrize("V", [7, 1000, 5003])
def test_ce_nan_rows_have_nan_statistics(T, V):
    """A diverged state shows in its token's lse, with a target and without, and in
    no other token's."""
    d = 64
    g = torch.Generator().manual_seed(T + V)
    Z, W = torch.randn(T, d, generator=g).to(BF), (torch.randn(V, d, generator=g) * 0.02).to(BF)
    targets = torch.randint(0, V, (T,), generator=g)
    targets[1] = targets[3] = -100
    want = ce_loss(Z, targets, W)
    bad = Z.clone()
    bad[1], bad[2] = float("nan"), float("nan")
    loss, lse, mean = ce_loss(bad, targets, W)
    rows = torch.zeros(T, dtype=torch.bool)
    rows[1] = rows[2] = True
    assert torch.equal(torch.isnan(lse).cpu(), rows)
    assert float(loss[1]) == 0 and math.isnan(float(loss[2])) and math.isnan(float(mean[0]))
    assert torch.equal(lse.cpu()[~rows], want[1].cpu()[~rows])
    assert torch.equal(loss.cpu()[~rows], want[0].cpu()[~rows])


@pytest.mark.parametrize("T", [5, 1100])
def test_ce_logits_of_minus_infinity_weigh_nothing(T):
    """Logits that pass fp32's range downwards (3e38 * -10): exp of them is 0, in a
    chunk of such words alone and beside others."""
    V, d = 700, 8
    Z, W = torch.zeros(T, d, dtype=BF), torch.zeros(V, d, dtype=BF)
    Z[:, 0] = 3e38
    low = torch.zeros(V, dtype=torch.bool)
    low[:32] = low[64:200] = low[690:] = True
    W[low, 0] = -10.0
    targets = torch.full((T,), 40)
    loss, lse, mean = ce_loss(Z, targets, W)
    # the others' logits are 0: log of their number, to fp32's rounding of a sum and a logarithm
    want = math.log(int((~low).sum()))
    assert float((f64(lse) - want).abs().max()) <= 16 * 2.0 ** -24 * want
    assert torch.equal(loss, lse)
    W[:, 0] = -10.0
    assert bool((ce_loss(Z, targets, W)[1] == -math.inf).all())


@pytest.mark.parametrize("packed", [True, False])
def test_attention_over_no_keys(packed):
    """max_k = 0 and no table of keys: every query sees nothing, forward and backward."""
    H, KH, hd, n = 2, 1, 64, 8
    rows = lambda m, heads: torch.randn(m, heads * hd, device="cuda").to(BF)
    q, k, v, do = rows(n, H), rows(0, KH), rows(0, KH), rows(n, H)
    o, dq, lse = torch.full_like(q, 7.0), torch.full_like(q, 7.0), torch.zeros(H, n, device="cuda")
    kw = dict(max_q=4, max_k=0)
    if packed:
        kw["cu_q"] = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    ws = torch.empty(qat.workspace_size(qat.QAT_OP_ATTN_BWD, H, hd, n, False), dtype=torch.uint8, device="cuda")
    qat.qat_attn_fwd(q, k, v, o, lse, H, KH, hd, **kw)
    qat.qat_attn_bwd(do, q, k, v, o, lse, dq, torch.empty_like(k), torch.empty_like(v), H, KH, hd, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert qat.device_error() == 0
    assert not o.any() and not dq.any() and bool((lse == -math.inf).all())


def test_workspaces_of_another_device_or_with_gaps_are_refused():
    T, V, d, H, hd = 8, 64, 64, 2, 64
    Z, t = torch.zeros(T, d, dtype=BF, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    q = qat.QWeight(torch.zeros(V, d, dtype=BF, device="cuda"), None, None, 8)
    loss, lse = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    rows = [torch.zeros(T, H * hd, dtype=BF, device="cuda") for _ in range(8)]
    stats = torch.zeros(H, T, device="cuda")
    n = 1 << 20
    before = qat.launch_count()
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n),
               torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        for call in (lambda: qat.qat_ce_fwd(Z, t, loss, lse, 8, qw=q, workspace=ws),
                     lambda: qat.qat_ce_bwd(Z, t, lse, 8, qw=q, dZ=torch.empty_like(Z), workspace=ws),
                     lambda: qat.qat_attn_bwd(*rows[:5], stats, *rows[5:], H, H, hd, max_q=T, workspace=ws)):
            with pytest.raises(qat.QatError) as e:
                call()
            assert e.value.code == qat.QAT_ERR_ARG
    assert qat.launch_count() == before


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_far_positions_against_exact_products(interleaved):
    """To positions of +-2^53: the fraction of a turn of position * freqs in whole numbers,
    where a product rounded to 64 bits is off by 1e-4 radians at 2^40 and by one at 2^53."""
    from fractions import Fraction
    from test_gpu_rope import PAIR
    heads, hd, rot = 2, 32, 24
    freqs, m = qat.rope_freqs(rot, scaling="yarn", factor=4.0, trained_len=1024)
    places = [s * (2 ** e + k) for e in (31, 36, 40, 46, 52) for k in (0, 12345, -77) for s in (1, -1)]
    places += [2 ** 53, -(2 ** 53)]
    x = torch.randn(len(places), heads * hd, generator=torch.Generator().manual_seed(2))
    y = torch.empty(len(places), heads * hd, device="cuda")
    qat.qat_rope(x.cuda(), y, heads, hd, freqs, positions=torch.tensor(places, device="cuda"), scale=m,
                 interleaved=interleaved)
    torch.cuda.synchronize()
    want = f64(x).reshape(-1, heads, hd).clone()
    tol = torch.zeros_like(want)
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    turn = torch.tensor([[float(Fraction(n) * Fraction(f) % 1) for f in freqs.tolist()] for n in places],
                        dtype=torch.float64) * 2 * math.pi
    c, s = m * turn.cos()[:, None], m * turn.sin()[:, None]
    u, v = want[..., a].clone(), want[..., b].clone()
    want[..., a], want[..., b] = u * c - v * s, u * s + v * c
    tol[..., a] = tol[..., b] = PAIR * m * (u.abs() + v.abs())
    tol += 2.0 ** -24 * want.abs()
    err = (f64(y).reshape(want.shape) - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("shape", [(130, 1024, 512), (1000, 40, 8), (5000, 1000, 256), (9000, 520, 72), (20000, 2001, 512),
                                   (12000, 4000, 512), (300, 257, 640)])
def test_ce_gradients_of_small_heads_have_the_same_bits(shape):
    """Heads whose output tiles leave most of the GPU idle: the tokens are split, and their
    parts added in one order, run after run, added to a gradient, and from raw words."""
    from test_gpu_cross_entropy import check, make, run, workspace
    T, V, d = shape
    c = make(T, V, d, seed=T, ignored=0.1)
    first = run(c, V, d)
    if T * V <= 6_000_000:
        check(c, V, d, first)
    base = torch.randn(V, d, device="cuda")
    sums = []
    for _ in range(6):
        got = run(c, V, d)
        assert torch.equal(got[3], first[3]) and torch.equal(got[4], first[4])
        acc = base.clone()
        qat.qat_ce_bwd(c["Zd"], c["td"], first[1], 8, qw=c["q"], gscale=first[2][1:], dW=acc, accumulate_dW=True,
                       workspace=workspace(qat.QAT_OP_CE_BWD, V, d, T))
        sums.append(acc)
    raw = torch.empty_like(base)
    qat.qat_ce_bwd(c["Zd"], c["td"], first[1], 8, W=c["W"].cuda(), gscale=first[2][1:], dW=raw,
                   workspace=workspace(qat.QAT_OP_CE_BWD, V, d, T, True))
    torch.cuda.synchronize()
    assert qat.device_error() == 0
    assert all(torch.equal(a, sums[0]) for a in sums) and torch.equal(raw, first[4])
    # base added first: 64 slabs at most in a piece, a half step of the running sum each
    pieces = -(-T // 256)
    allowed = 2.0 ** -24 * (64 * pieces + 1) * (base.abs().max() + 64 * first[4].abs().max())
    assert float((sums[0] - base - first[4]).abs().max()) <= float(allowed)
