"""The language-model operators as the library's own paths run them: the
depth-recurrent core with attention and rotary positions, the tied head's step
on its cross entropy, and both in one training step -- against float64
autograd of the same composition on the CPU."""
import numpy as np
import pytest
import torch

from lm_reference import f64
from quantization_aware_tiny_b200 import qat, steps
from quantization_aware_tiny_b200 import synthetic as sy

pytestmark = pytest.mark.gpu

# Every tensor handed on is rounded to bf16, at most half a step (2^-8) each; the
# float64 side rounds nowhere.  Independent roundings add in squares: one
# application has 8 in the forward (qkv, rotation, P, att, x1, pre / h, x) and 8 in
# the backward (dpre, dx1, datt, P, dS, dqkv, rotation, dx), so its results are off
# by at most sqrt(16 R) * 2^-8 relative to their norm.
STEP = 2.0 ** -8


def bound(R):
    return (16 * R) ** 0.5 * STEP


def fro(got, ref):
    return float((f64(got) - ref).norm() / ref.norm())


def heads_out(qkv, H, KH, hd, lens, rope, pos, window):
    """Float64 attention of rotated Q|K|V rows (torch operations, for autograd)."""
    T = qkv.shape[0]
    x = qkv.reshape(T, H + 2 * KH, hd)
    qk, v = x[:, :H + KH], x[:, H + KH:]
    if rope is not None:
        fr, m = f64(rope[0]), rope[1]
        ang = pos.double()[:, None] * fr[None] * 2 * np.pi
        c, s = m * ang.cos()[:, None], m * ang.sin()[:, None]
        n = fr.numel()
        a, b = qk[..., :n], qk[..., n:2 * n]
        qk = torch.cat([a * c - b * s, a * s + b * c, qk[..., 2 * n:]], -1)
    out, at = [], 0
    for n in lens:
        r = slice(at, at + n)
        at += n
        q, k = qk[r, :H], qk[r, H:].repeat_interleave(H // KH, 1)
        w = v[r].repeat_interleave(H // KH, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) / hd ** 0.5
        keep = torch.ones(n, n, dtype=torch.bool).tril()
        if window:
            keep = keep.triu(1 - window)
        p = torch.softmax(s.masked_fill(~keep, -float("inf")), -1)
        out.append(torch.einsum("hij,jhd->ihd", p, w).reshape(n, H * hd))
    return torch.cat(out)


def reference_core(core, x, R, lens, pos, window):
    """States through R applications from the core's own operands, with gradients."""
    ops = [f64(q.operand).requires_grad_() for q in (core.q_qkv, core.q_o, core.q_fc, core.q_proj)]
    a = core.attention
    x = x.clone().requires_grad_()
    y = x
    for _ in range(R):
        att = heads_out(y @ ops[0].T, a.heads, a.kv_heads, core.hd, lens, a.rope, pos, window)
        x1 = y + att @ ops[1].T
        y = x1 + (torch.relu(x1 @ ops[2].T) ** 2) @ ops[3].T
    return x, y, ops


def make_core(d, H, KH, hidden, T, attention, seed=0):
    c = sy.recurrent_core_case(d=d, H=hidden, T=T, seed=seed)
    kv = KH * (d // H)
    g = {k: torch.from_numpy(c[k]).cuda() for k in ("Wq", "Wo", "Wfc", "Wproj")}
    rng = torch.Generator().manual_seed(seed + 11)
    g.update({k: (torch.randn(kv, d, generator=rng) * sy.W_STD).cuda() for k in ("Wk", "Wv")})
    return steps.RecurrentCore(*(g[k] for k in ("Wq", "Wk", "Wv", "Wo", "Wfc", "Wproj")), bits=6,
                               attention=attention), c["X"]


@pytest.mark.parametrize("R,window,packed", [(1, 0, False), (2, 0, True), (1, 40, True)])
def test_core_with_attention(R, window, packed):
    """d = 160, 4 query heads over 2 of 40; equal and packed sequences."""
    d, H, KH = 160, 4, 2
    lens = [150, 1, 77] if packed else [76, 76, 76]
    T = sum(lens)
    pos = torch.cat([torch.arange(n) for n in lens])
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda") if packed else None
    att = steps.CoreAttention(H, KH, max(lens), cu=cu, window=window, rope=qat.rope_freqs(24),
                              positions=pos.cuda() if packed else None)
    core, X = make_core(d, H, KH, 320, T, att)
    dY = sy.act_bf16(np.random.default_rng(1), T, d, std=sy.DY_STD)
    out = core.forward_train(X.cuda(), R).clone()
    dX = core.backward(dY.cuda())
    again = core.forward(X.cuda().clone(), R)
    torch.cuda.synchronize()
    assert qat.device_error() == 0
    assert torch.equal(out, again)  # the inference path runs the same kernels
    x, y, ops = reference_core(core, f64(X), R, lens, pos, window)
    y.backward(f64(dY))
    assert fro(out, y.detach()) <= bound(R)
    assert fro(dX, x.grad) <= bound(R)
    for name, got, op in zip(("dWqkv", "dWo", "dWfc", "dWproj"),
                             (core.dWqkv, core.dWo, core.dWfc, core.dWproj), ops):
        assert fro(got, op.grad) <= bound(R), name


@pytest.mark.parametrize("own_stream", [False, True])
def test_core_rows_behind_the_last_sequence(own_stream):
    """A packed batch that does not fill its rows, in buffers that held NaN: the rows
    behind it attend to nothing, and every weight gradient is that of the composition."""
    d, H, KH, R = 160, 4, 2, 2
    lens, tail = [100, 33], 27
    T = sum(lens) + tail
    pos = torch.cat([torch.arange(n) for n in lens + [tail]])
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    att = steps.CoreAttention(H, KH, max(lens), cu=cu, rope=qat.rope_freqs(24), positions=pos.cuda())
    core, X = make_core(d, H, KH, 320, T, att)
    dY = sy.act_bf16(np.random.default_rng(1), T, d, std=sy.DY_STD)
    tb = core._train_buffers(T, R, "cuda")
    for n in ("att", "dqkv"):
        tb[n].fill_(float("nan"))
    x, dy = X.cuda(), dY.cuda()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if own_stream else None
    out = core.forward_train(x, R, stream=stream)
    dX = core.backward(dy, stream=stream)
    torch.cuda.synchronize()
    assert qat.device_error() == 0
    kept = out.clone()
    core.forward(x.clone(), R)
    core._att[0].fill_(float("nan"))
    again = core.forward(x.clone(), R)
    torch.cuda.synchronize()
    assert torch.equal(kept, again)
    n = sum(lens)
    ops = [f64(q.operand).requires_grad_() for q in (core.q_qkv, core.q_o, core.q_fc, core.q_proj)]
    xr = f64(X).requires_grad_()
    y = xr
    for _ in range(R):
        a = heads_out((y @ ops[0].T)[:n], H, KH, core.hd, lens, att.rope, pos[:n], 0)
        x1 = y + torch.cat([a, a.new_zeros(tail, d)]) @ ops[1].T
        y = x1 + (torch.relu(x1 @ ops[2].T) ** 2) @ ops[3].T
    y.backward(f64(dY))
    assert fro(kept, y.detach()) <= bound(R)
    assert fro(dX, xr.grad) <= bound(R)
    for name, got, op in zip(("dWqkv", "dWo", "dWfc", "dWproj"),
                             (core.dWqkv, core.dWo, core.dWfc, core.dWproj), ops):
        assert fro(got, op.grad) <= bound(R), name


def test_core_backward_application_and_accumulate_with_attention():
    d, H, KH, T = 160, 4, 4, 130
    att = steps.CoreAttention(H, KH, 65, rope=qat.rope_freqs(40))
    core, X = make_core(d, H, KH, 320, T, att)
    dY = sy.act_bf16(np.random.default_rng(1), T, d, std=sy.DY_STD).cuda()
    core.forward_train(X.cuda(), 1)
    dX = core.backward(dY).clone()
    w = [t.clone() for t in (core.dWqkv, core.dWo, core.dWfc, core.dWproj)]
    dx = torch.empty_like(dX)
    core.backward_application(core._saved(0), dY, dx, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(dx, dX)
    for a, b in zip((core.dWqkv, core.dWo, core.dWfc, core.dWproj), w):
        # the same sum twice, in fp32, its parts in any order
        assert float((a - 2 * b).abs().max()) <= 64 * 2 ** -24 * float(b.abs().max())


def test_core_refuses_head_counts_that_do_not_fit():
    with pytest.raises(ValueError):
        make_core(160, 4, 2, 320, 8, steps.CoreAttention(4, 4, 8))
    with pytest.raises(ValueError):
        steps.CoreAttention(4, 2, 8, cu=torch.zeros(2, dtype=torch.int32), rope=(None, 1.0))


def test_head_step_on_its_cross_entropy():
    """step_loss against float64 autograd through head and MLP; the gradients equal
    step()'s on the gradient that the loss sends to the logits."""
    T, V, d, hidden = 300, 1000, 128, 256
    c = sy.head_mlp_case(T=T, vocab=V, d=d, H=hidden)
    t = {k: torch.from_numpy(c[k]).cuda() for k in ("Wemb", "Wfc", "Wproj")}
    s = steps.HeadMlpStep(t["Wemb"], t["Wfc"], t["Wproj"], T, logits=False)
    targets = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(0))
    targets[::7] = -100
    mean = s.step_loss(c["X"].cuda(), targets.cuda())
    torch.cuda.synchronize()
    x = f64(c["X"]).requires_grad_()
    we, wf, wp = (f64(q.operand).requires_grad_() for q in s.q)
    z = (torch.relu(x @ wf.T) ** 2) @ wp.T
    loss = torch.nn.functional.cross_entropy(z @ we.T, targets)
    loss.backward()
    # pre, h, Z, g, dZ, dpre, dX: 7 roundings
    assert abs(float(mean) - float(loss.detach())) <= 7 ** 0.5 * STEP * float(loss.detach())
    for name, got, ref in (("dX", s.dX, x.grad), ("dWemb", s.dWemb, we.grad), ("dWfc", s.dWfc, wf.grad),
                           ("dWproj", s.dWproj, wp.grad)):
        assert fro(got, ref) <= 7 ** 0.5 * STEP, name


def test_core_into_head_trains_in_a_graph():
    """Rotary, attention, the core's linears and the head's loss as one captured
    training step, replayed on new words; against float64 autograd."""
    T, V, d, H, KH = 192, 520, 160, 4, 2
    att = steps.CoreAttention(H, KH, 64, rope=qat.rope_freqs(40))
    core, X = make_core(d, H, KH, 320, T, att)
    Wemb = torch.randn(V, d, generator=torch.Generator().manual_seed(3)) * 0.02
    q = qat.quantize_weight(Wemb.cuda(), 8)
    x, words = X.cuda(), torch.zeros(T, dtype=torch.int64, device="cuda")
    loss, lse, mean = (torch.empty(n, device="cuda") for n in (T, T, 2))
    dZ, dW = torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(V, d, device="cuda")
    ws = torch.empty(qat.workspace_size(qat.QAT_OP_CE_BWD, V, d, T, False), dtype=torch.uint8, device="cuda")

    def step():
        z = core.forward_train(x, 1)
        qat.qat_ce_fwd(z, words, loss, lse, 8, qw=q, mean=mean, workspace=ws)
        qat.qat_ce_bwd(z, words, lse, 8, qw=q, gscale=mean[1:], dZ=dZ, dW=dW, workspace=ws)
        return core.backward(dZ)

    step()
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        dX = step()
    words.copy_(torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(4)))
    words[5] = -1
    graph.replay()
    torch.cuda.synchronize()
    assert qat.device_error() == 0
    xr, y, ops = reference_core(core, f64(X), 1, [64, 64, 64], torch.arange(T) % 64, 0)
    we = f64(q.operand).requires_grad_()
    ref = torch.nn.functional.cross_entropy(y @ we.T, words.cpu(), ignore_index=-1)
    ref.backward()
    assert abs(float(mean[0]) - float(ref.detach())) <= bound(1) * float(ref.detach())
    for name, got, r in (("dX", dX, xr.grad), ("dWemb", dW, we.grad), ("dWqkv", core.dWqkv, ops[0].grad),
                         ("dWo", core.dWo, ops[1].grad), ("dWfc", core.dWfc, ops[2].grad),
                         ("dWproj", core.dWproj, ops[3].grad)):
        assert fro(got, r) <= bound(1), name
