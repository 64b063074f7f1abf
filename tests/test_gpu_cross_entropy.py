"""Softmax cross entropy of the QAT head on the GPU against the float64 form:
loss, log-sum-exp, mean, dZ and dW, element by element."""
import pytest
import torch

from lm_reference import cross_entropy, f64, within
from quantization_aware_tiny_b200 import qat

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


def make(T, V, d, seed=0, ignored=0.0, lean=8.0, ldz=None):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(V, d, generator=g) * 0.02
    targets = torch.randint(0, V, (T,), generator=g)
    Z = torch.randn(T, d, generator=g)
    Z = (Z + lean * torch.rand(T, 1, generator=g) * W[targets] / (0.02 * d ** 0.5)).to(BF)
    targets[torch.rand(T, generator=g) < ignored] = -100
    q = qat.quantize_weight(W.cuda(), 8)
    wide = torch.full((T, ldz or d), float("nan"), dtype=BF)
    wide[:, :d] = Z
    return {"W": W, "Z": Z, "t": targets, "q": q, "Zd": wide.cuda()[:, :d], "td": targets.cuda()}


def outputs(T, V, d):
    e = lambda *s, dt=F32: torch.full(s, float("nan"), dtype=dt, device="cuda")
    return e(T), e(T), e(2), e(T, d, dt=BF), e(V, d)


def workspace(op, V, d, T, raw=False):
    return torch.empty(qat.workspace_size(op, V, d, T, raw), dtype=torch.uint8, device="cuda")


def run(c, V, d, dloss=None, use_mean=True, ws=None):
    T = c["t"].shape[0]
    loss, lse, mean, dZ, dW = outputs(T, V, d)
    ws = workspace(qat.QAT_OP_CE_BWD, V, d, T) if ws is None else ws
    qat.qat_ce_fwd(c["Zd"], c["td"], loss, lse, 8, qw=c["q"], mean=mean,
                   workspace=workspace(qat.QAT_OP_CE_FWD, V, d, T))
    qat.qat_ce_bwd(c["Zd"], c["td"], lse, 8, qw=c["q"], dloss=dloss,
                   gscale=mean[1:] if use_mean else None, dZ=dZ, dW=dW, workspace=ws)
    torch.cuda.synchronize()
    assert qat.device_error() == 0
    return loss, lse, mean, dZ, dW


def check(c, V, d, got, dloss=None, use_mean=True):
    loss, lse, mean, dZ, dW = got
    w, z = f64(c["q"].operand), f64(c["Z"])
    n = int(((c["t"] >= 0) & (c["t"] < V)).sum())
    r = cross_entropy(z, w, c["t"], dloss, (1.0 / n if n else 0.0) if use_mean else 1.0)
    within(loss, r["loss"], r["loss_tol"], "loss")
    within(lse, r["lse"], r["lse_tol"], "lse")
    within(dZ, r["dZ"], r["dZ_tol"], "dZ")
    within(dW, r["dW"], r["dW_tol"], "dW")
    tol = float(r["loss_tol"].max()) + 2 ** -22 * abs(r["mean"])
    assert abs(float(mean[0]) - r["mean"]) <= tol
    assert float(mean[1]) == pytest.approx(1.0 / n if n else 0.0, rel=2 ** -23)


SHAPES = [(1, 8, 8), (1, 1, 64), (3, 7, 8), (31, 33, 72), (128, 160, 64), (255, 1024, 512), (256, 1000, 128),
          (257, 1023, 136), (300, 129, 512), (700, 257, 640), (513, 2049, 256)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("ignored", [0.0, 0.2])
def test_ce_against_float64(shape, ignored):
    """Token tails, vocabularies of one word, odd and just past a tile, widths off 64."""
    T, V, d = shape
    c = make(T, V, d, seed=T + V + d, ignored=ignored)
    check(c, V, d, run(c, V, d))


@pytest.mark.parametrize("T", [5, 600])
def test_ce_every_row_ignored(T):
    """No counted token: loss, mean and every gradient are zero, not NaN."""
    V, d = 264, 64
    c = make(T, V, d, ignored=0.0)
    c["t"] = torch.full((T,), -100)
    c["t"][::2] = V  # just past the vocabulary counts for nothing as well
    c["td"] = c["t"].cuda()
    got = run(c, V, d)
    check(c, V, d, got)
    assert float(got[2][0]) == 0 and float(got[2][1]) == 0
    assert not got[3].any() and not got[4].any()


def test_ce_upstream_gradient_per_token():
    T, V, d = 333, 515, 128
    c = make(T, V, d, ignored=0.1)
    dloss = torch.randn(T, generator=torch.Generator().manual_seed(3))
    got = run(c, V, d, dloss=dloss.cuda(), use_mean=False)
    check(c, V, d, got, dloss=dloss, use_mean=False)


def test_ce_strided_rows_beside_nan():
    """Z as a column range of wider rows whose other columns hold NaN."""
    T, V, d = 300, 600, 72
    c = make(T, V, d, ldz=136)
    check(c, V, d, run(c, V, d))


@pytest.mark.parametrize("scale", [0.0, 60.0])
def test_ce_flat_and_peaked(scale):
    """All logits equal, and a softmax that is one to fp32's last bits."""
    T, V, d = 260, 300, 64
    c = make(T, V, d, lean=scale)
    if scale == 0.0:
        c["Z"] = torch.zeros_like(c["Z"])
        c["Zd"] = c["Z"].cuda()
    check(c, V, d, run(c, V, d))


def test_ce_small_workspace_gives_more_pieces():
    """Down to one row tile a piece; below that the call refuses."""
    T, V, d = 1000, 520, 128
    c = make(T, V, d, ignored=0.1)
    one = 256 * 520 * 4 + 1024
    for size in (one, one * 2 + 100, one * 3):
        check(c, V, d, run(c, V, d, ws=torch.empty(size, dtype=torch.uint8, device="cuda")))
    dZ, lse = torch.zeros(T, d, dtype=BF, device="cuda"), torch.zeros(T, device="cuda")
    with pytest.raises(qat.QatError) as e:
        qat.qat_ce_bwd(c["Zd"], c["td"], lse, 8, qw=c["q"], dZ=dZ,
                       workspace=torch.empty(one - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.code == qat.QAT_ERR_WORKSPACE


def test_ce_raw_weight_equals_prequantized():
    T, V, d = 300, 1000, 128
    c = make(T, V, d)
    a = run(c, V, d)
    loss, lse, mean, dZ, dW = outputs(T, V, d)
    ws = workspace(qat.QAT_OP_CE_BWD, V, d, T, True)
    Wd = c["W"].cuda()
    qat.qat_ce_fwd(c["Zd"], c["td"], loss, lse, 8, W=Wd, mean=mean, workspace=ws)
    qat.qat_ce_bwd(c["Zd"], c["td"], lse, 8, W=Wd, gscale=mean[1:], dZ=dZ, dW=dW, workspace=ws)
    torch.cuda.synchronize()
    for x, y in zip(a[:4], (loss, lse, mean, dZ)):
        assert torch.equal(x, y)


def test_ce_one_gradient_only_and_accumulate():
    T, V, d = 300, 264, 64
    c = make(T, V, d)
    loss, lse, mean, dZ, dW = run(c, V, d)
    ws = workspace(qat.QAT_OP_CE_BWD, V, d, T)
    only = torch.full_like(dZ, float("nan"))
    qat.qat_ce_bwd(c["Zd"], c["td"], lse, 8, qw=c["q"], gscale=mean[1:], dZ=only, workspace=ws)
    base = torch.randn(V, d, device="cuda")
    acc = base.clone()
    qat.qat_ce_bwd(c["Zd"], c["td"], lse, 8, qw=c["q"], gscale=mean[1:], dW=acc, accumulate_dW=True,
                   workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(only, dZ)
    # three fp32 additions (two halves, the base), each off by half a step of the sums around it
    assert float((acc - base - dW).abs().max()) <= 4 * 2 ** -24 * float(base.abs().max() + 1)


def test_ce_empty_batch():
    V, d = 264, 64
    c = make(4, V, d)
    z, t = c["Zd"][:0], c["td"][:0]
    mean, dW = torch.ones(2, device="cuda"), torch.ones(V, d, device="cuda")
    e = torch.empty(0, device="cuda")
    qat.qat_ce_fwd(z, t, e, e, 8, qw=c["q"], mean=mean)
    qat.qat_ce_bwd(z, t, e, 8, qw=c["q"], dW=dW, accumulate_dW=True)
    torch.cuda.synchronize()
    assert not mean.any() and bool((dW == 1).all())
    qat.qat_ce_bwd(z, t, e, 8, qw=c["q"], dW=dW)
    torch.cuda.synchronize()
    assert not dW.any()


def test_ce_gradient_against_differences():
    """dZ along a random direction against the loss's own difference quotient
    (float64 form at both ends: the GPU's part is the gradient)."""
    T, V, d = 64, 200, 64
    c = make(T, V, d)
    loss, lse, mean, dZ, dW = run(c, V, d)
    z, w = f64(c["Z"]), f64(c["q"].operand)
    g = torch.Generator().manual_seed(9)
    dirz, dirw, h = torch.randn(T, d, generator=g).double(), torch.randn(V, d, generator=g).double(), 1e-5
    f = lambda a, b: cross_entropy(a, b, c["t"])["mean"]
    r = cross_entropy(z, w, c["t"], None, 1.0 / T)
    for got, dirn, plus, minus, tol in (
            (dZ, dirz, f(z + h * dirz, w), f(z - h * dirz, w), r["dZ_tol"]),
            (dW, dirw, f(z, w + h * dirw), f(z, w - h * dirw), r["dW_tol"])):
        quotient = (plus - minus) / (2 * h)
        allowed = float((tol * dirn.abs()).sum()) + 1e-8
        assert abs(float((f64(got) * dirn).sum()) - quotient) <= allowed


def test_ce_same_bits_every_time_and_in_a_graph():
    """Loss and dZ have the same bits in every run; a captured training call
    replays on new inputs while eager calls use the same entry points."""
    T, V, d = 520, 1000, 128
    c, c2 = make(T, V, d, seed=1), make(T, V, d, seed=2)
    a, b = run(c, V, d), run(c, V, d)
    for x, y in zip(a[:4], b[:4]):
        assert torch.equal(x, y)
    Z, t = c["Zd"].clone(), c["td"].clone()
    loss, lse, mean, dZ, dW = outputs(T, V, d)
    ws = workspace(qat.QAT_OP_CE_BWD, V, d, T)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        qat.qat_ce_fwd(Z, t, loss, lse, 8, qw=c["q"], mean=mean, workspace=ws)
        qat.qat_ce_bwd(Z, t, lse, 8, qw=c["q"], gscale=mean[1:], dZ=dZ, dW=dW, workspace=ws)
    for src in (c2, c):
        Z.copy_(src["Zd"])
        t.copy_(src["td"])
        graph.replay()
        eager = run({**src, "q": c["q"]}, V, d)
        for x, y in zip(eager[:4], (loss, lse, mean, dZ)):
            assert torch.equal(x, y)


def test_ce_refusals():
    V, d, T = 64, 64, 8
    c = make(T, V, d)
    loss, lse, mean, dZ, dW = outputs(T, V, d)
    ws = workspace(qat.QAT_OP_CE_BWD, V, d, T)
    ok = dict(qw=c["q"], mean=mean, workspace=ws)

    def bad(code, *a, **k):
        with pytest.raises(qat.QatError) as e:
            qat.qat_ce_fwd(*a, **k)
        assert e.value.code == code

    before = qat.launch_count()
    bad(qat.QAT_ERR_ARG, c["Zd"], c["td"].int(), loss, lse, 8, **ok)
    bad(qat.QAT_ERR_ARG, c["Zd"].float(), c["td"], loss, lse, 8, **ok)
    bad(qat.QAT_ERR_ARG, c["Zd"], c["td"][:4], loss, lse, 8, **ok)
    bad(qat.QAT_ERR_ARG, c["Zd"], c["t"], loss, lse, 8, **ok)
    bad(qat.QAT_ERR_ARG, c["Zd"], c["td"], loss, lse, 7, **ok)
    bad(qat.QAT_ERR_ARG, c["Zd"], c["td"], torch.empty(2 * T, device="cuda")[::2], lse, 8, **ok)
    bad(qat.QAT_ERR_ARG, c["Zd"], c["td"], loss, lse, 8, workspace=ws)
    bad(qat.QAT_ERR_ARG, c["Zd"][:, :32], c["td"], loss, lse, 8, **ok)
    bad(qat.QAT_ERR_ARG, c["Zd"].t().contiguous().t(), c["td"], loss, lse, 8, **ok)
    bad(qat.QAT_ERR_WORKSPACE, c["Zd"], c["td"], loss, lse, 8, qw=c["q"])
    bad(qat.QAT_ERR_WORKSPACE, c["Zd"], c["td"], loss, lse, 8, qw=c["q"], workspace=ws[:64])
    bad(qat.QAT_ERR_ALIGN, c["Zd"], c["td"], loss, lse, 8, qw=c["q"], workspace=ws[8:])
    assert qat.launch_count() == before


def test_ce_long_sum_over_tokens():
    """More tokens than one accumulator sums: dW's runs are added in order, so the
    bits repeat where the output tiles alone fill the GPU (no parallel split)."""
    T, V, d = 5000, 5120, 512
    c = make(T, V, d, ignored=0.05)
    a, b = run(c, V, d), run(c, V, d)
    check(c, V, d, a)
    assert torch.equal(a[4], b[4])


@pytest.mark.parametrize("shape", [(1, 20001, 264), (40, 9000, 64), (300, 20001, 136), (1000, 5003, 512)])
def test_ce_few_tokens_of_many_words(shape):
    """dZ's reduction over the vocabulary is split and joined in order: the formula's
    values, the same bits twice, and with a workspace that has no room for the parts."""
    T, V, d = shape
    c = make(T, V, d, seed=T, ignored=0.1 if T > 1 else 0.0)
    got = run(c, V, d)
    check(c, V, d, got)
    assert all(torch.equal(a, b) for a, b in zip(got[:4], run(c, V, d)[:4]))
    small = torch.empty(4 * T * ((V + 7) // 8 * 8) + 4 * T + 1024, dtype=torch.uint8, device="cuda")
    assert small.numel() < qat.workspace_size(qat.QAT_OP_CE_BWD, V, d, T, False)
    check(c, V, d, run(c, V, d, ws=small))


@pytest.mark.parametrize("T", [1000, 1100])
def test_ce_runs_of_tokens_added_in_order(T):
    """As many output tiles as fill the GPU: dW's runs of tokens are added by one CTA
    pair, the first written over what was there; the same bits twice."""
    V, d = 10008, 256
    c = make(T, V, d, seed=T, ignored=0.1)
    got = run(c, V, d)
    check(c, V, d, got)
    assert torch.equal(got[4], run(c, V, d)[4])
    dW = got[4].clone()
    ws = workspace(qat.QAT_OP_CE_BWD, V, d, T)
    qat.qat_ce_bwd(c["Zd"], c["td"], got[1], 8, qw=c["q"], gscale=got[2][1:], dW=dW, accumulate_dW=True, workspace=ws)
    torch.cuda.synchronize()
    # the runs (at most 2, each within twice the largest sum M) added to the first sum: adds
    # of at most M, 3 M and 2 M, each off by at most half a step, 2^-24
    assert bool(((dW - 2 * got[4]).abs() <= 6 * 2 ** -24 * got[4].abs().max()).all())
