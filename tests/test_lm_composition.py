"""The recurrent core with attention where attention matters: scores spread over
more than one, heads whose term is as large as the residual, Q, K and V blocks and
the attention's own terms compared one by one.

Bounds: the composition with the library's roundings (lm_composition.run with r =
bf16) against the exact one, twice.  The library rounds the same values at the same
places, so its deviation is a sample of the same size; its fp32 sums add 2^-16 of a
rounding.  The CPU tests show that a composition that is wrong somewhere is farther
off than that.
"""
import math

import pytest
import torch

import lm_composition as lc
from lm_reference import f64

BF = torch.bfloat16

# d, query heads, key heads, head size, MLP, R, window, sequences (None: equal ones), rows behind, rotary
CASES = {
    "equal": (160, 4, 2, 40, 320, 1, 0, [76] * 3, 0, 24),
    "packed, two applications": (160, 4, 2, 40, 320, 2, 0, [150, 1, 77], 0, 24),
    "packed, window, rows behind": (160, 4, 2, 40, 320, 1, 40, [150, 1, 77], 27, 24),
    "wide heads of one key head": (96, 4, 1, 64, 192, 1, 0, [130, 60], 0, 64),
    "narrow heads that share nothing": (192, 3, 3, 32, 384, 2, 0, [129, 40], 0, 32),
}


def weights(case):
    """Weights in fp32 with queries and keys scaled so that scores have a spread of about
    1.5, values and outputs so that attention's term is about as large as the state."""
    d, H, KH, hd, hidden = CASES[case][:5]
    g = torch.Generator().manual_seed(sorted(CASES).index(case))
    w = lambda n, k, std: torch.randn(n, k, generator=g) * std
    qk = (1.5 ** 0.5) / d ** 0.5
    return (w(H * hd, d, qk), w(KH * hd, d, qk), w(KH * hd, d, 1.5 / d ** 0.5), w(d, H * hd, 1.5 / (H * hd) ** 0.5),
            w(hidden, d, 0.7 / d ** 0.5), w(d, hidden, 0.5 / hidden ** 0.5))


def inputs(case):
    d, lens, tail = CASES[case][0], CASES[case][7], CASES[case][8]
    g = torch.Generator().manual_seed(17)
    T = sum(lens) + tail
    return torch.randn(T, d, generator=g).to(BF), (torch.randn(T, d, generator=g) * 1e-2).to(BF)


def places(case):
    lens, tail = CASES[case][7], CASES[case][8]
    return torch.cat([torch.arange(n) for n in lens + ([tail] if tail else [])])


def attention(case, freqs):
    d, H, KH, hd, hidden, R, window, lens, tail, rotary = CASES[case]
    return lc.Attention(H, KH, hd, lens, window, freqs, 1.0, places(case))


def plain_freqs(rotary):
    return 10000.0 ** (-2.0 * torch.arange(rotary // 2, dtype=torch.float64) / rotary) / (2 * math.pi)


def operands(case):
    """The weights as the library would round them, near enough for its noise: bf16."""
    w = [lc.bf16(t.double()) for t in weights(case)]
    return [torch.cat(w[:3])] + w[3:]


@pytest.mark.parametrize("case", CASES)
def test_written_out_backward_is_autograd(case):
    ops = [w.requires_grad_() for w in operands(case)]
    att, R = attention(case, plain_freqs(CASES[case][9])), CASES[case][5]
    x, dY = (t.double() for t in inputs(case))
    x.requires_grad_()
    y = x
    for _ in range(R):
        q, k, v = att.columns(y @ ops[0].T)
        q, k = att.turn(q, False), att.turn(k, False)
        heads = torch.zeros(x.shape[0], att.heads * att.hd, dtype=torch.float64)
        for rows, c, ck in att.pairs():
            heads = heads.index_put((torch.arange(rows.start, rows.stop)[:, None],
                                     torch.arange(c.start, c.stop)[None]),
                                    att.probabilities(q[rows, c], k[rows, ck], None) @ v[rows, ck])
        y1 = y + heads @ ops[1].T
        y = y1 + (torch.relu(y1 @ ops[2].T) ** 2) @ ops[3].T
    y.backward(dY)
    got = lc.run(att, [w.detach() for w in ops], x.detach(), dY, R)
    q, k = att.heads * att.hd, (att.heads + att.kv_heads) * att.hd
    want = dict(out=y.detach(), dX=x.grad, dWq=ops[0].grad[:q], dWk=ops[0].grad[q:k], dWv=ops[0].grad[k:],
                dWo=ops[1].grad, dWfc=ops[2].grad, dWproj=ops[3].grad)
    assert max(lc.off(got, want).values()) < 1e-12


def bounds(att, ops, x, dY, R):
    want = lc.run(att, ops, x, dY, R)
    noise = lc.off(lc.run(att, ops, x, dY, R, lc.bf16), want)
    return want, {n: 2 * v + 2.0 ** -24 for n, v in noise.items()}


@pytest.mark.parametrize("case", CASES)
def test_broken_compositions_are_seen(case):
    """Every wrong composition passes the bound of some result at least fourfold, a fifth of
    dQ or dK missing among them, and the scores are no flat ones."""
    d, H, KH, hd, hidden, R, window, lens, tail, rotary = CASES[case]
    ops, att = operands(case), attention(case, plain_freqs(rotary))
    x, dY = (t.double() for t in inputs(case))
    want, allowed = bounds(att, ops, x, dY, R)
    q, k = att.forward(x @ ops[0].T, lc.exact)[0]
    rows, c, ck = next(att.pairs())
    assert 1.0 < float((q[rows, c] @ k[rows, ck].T / hd ** 0.5).std()) < 4.0
    assert max(allowed.values()) < 0.08
    for broken in lc.BROKEN:
        if (broken == "no window" and not window) or (broken.startswith("one head") and H == KH):
            continue
        wrong = lc.off(lc.run(att, ops, x, dY, R, lc.exact, broken), want)
        excess = {n: wrong[n] / allowed[n] for n in wrong}
        worst = max(excess, key=excess.get)
        assert excess[worst] > 4, (broken, worst, excess)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_core_against_the_exact_composition(case):
    """States, the attention's own terms forward and backward, dX, and every block of the
    weights' gradients."""
    from quantization_aware_tiny_b200 import qat, steps
    d, H, KH, hd, hidden, R, window, lens, tail, rotary = CASES[case]
    cu = None
    if len(set(lens)) > 1 or tail:
        cu = torch.tensor([sum(lens[:n]) for n in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    freqs, m = qat.rope_freqs(rotary)
    core = steps.RecurrentCore(*(w.cuda() for w in weights(case)), bits=6, attention=steps.CoreAttention(
        H, KH, max(lens), cu=cu, window=window, rope=(freqs, m), positions=places(case).cuda() if cu is not None else None))
    x, dY = inputs(case)
    out = core.forward_train(x.cuda(), R).clone()
    dX = core.backward(dY.cuda())
    torch.cuda.synchronize()
    assert qat.device_error() == 0
    tb = core._tb
    got = dict(out=f64(out), dX=f64(dX), dWo=f64(core.dWo), dWfc=f64(core.dWfc), dWproj=f64(core.dWproj))
    q, k = H * hd, (H + KH) * hd
    got.update(dWq=f64(core.dWqkv[:q]), dWk=f64(core.dWqkv[q:k]), dWv=f64(core.dWqkv[k:]))
    for n in range(R):
        got["attended %d" % n] = f64(tb["x1"][n]) - f64(tb["states"][n])
        got["sent %d" % n] = f64(tb["g"][n - 1] if n else dX) - f64(tb["dx1"][n])
    ops = [f64(o.operand) for o in (core.q_qkv, core.q_o, core.q_fc, core.q_proj)]
    want, allowed = bounds(attention(case, f64(freqs)), ops, x.double(), dY.double(), R)
    assert sorted(got) == sorted(want)
    wrong = lc.off(got, want)
    assert all(wrong[n] <= allowed[n] for n in want), {n: (wrong[n], allowed[n]) for n in want}
