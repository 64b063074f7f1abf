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
