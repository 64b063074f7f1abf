"""Rotary positions on the GPU against the float64 rotation."""
import math

import pytest
import torch

from lm_reference import E, U, f64, rotate, within
from quantization_aware_tiny_b200 import qat

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# the angle's rounding to fp32 (2 pi of 2^-25 turns: 3.2 E), sine and cosine (2 E each,
# scaled: 1 E more), two products and a sum: 10 E of the pair's magnitude, rounded up
PAIR = 12 * E


def check(T, heads, head_dim, rotary, dtype, interleaved, inverse, far=0, pad=0, in_place=False,
          seq_len=0, scale=1.0, freqs=None, given=True):
    g = torch.Generator().manual_seed(T + heads + head_dim + rotary)
    W = heads * head_dim
    x = torch.randn(T, W, generator=g).to(dtype)
    wide = torch.full((T, W + pad), float("nan"), dtype=dtype)
    wide[:, :W] = x
    pos = torch.randint(0, far + 1, (T,), generator=g) if given else None
    freqs = qat.rope_freqs(rotary)[0] if freqs is None else freqs
    xd = wide.cuda()
    yd = xd if in_place else torch.full((T + 1, W + 2 * pad), 7.0, dtype=dtype, device="cuda")
    qat.qat_rope(xd[:, :W], yd[:T, :W], heads, head_dim, freqs, positions=None if pos is None else pos.cuda(),
                 seq_len=seq_len, interleaved=interleaved, scale=scale, inverse=inverse)
    torch.cuda.synchronize()
    at = pos if given else (torch.arange(T) % seq_len if seq_len else torch.arange(T))
    ref, mag = rotate(f64(x), heads, head_dim, f64(freqs), at, interleaved, scale, inverse)
    tol = PAIR * mag + (U if dtype == BF else E) * ref.abs()
    within(yd[:T, :W], ref, tol, "rotated")
    if in_place:
        assert bool(torch.isnan(yd[:, W:]).all())
    else:  # what lies beside and behind the rows stays
        assert bool((yd[:T, W:] == 7).all()) and bool((yd[T] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dims", [(64, 64), (80, 80), (64, 16), (64, 2), (64, 6), (8, 8), (8, 4), (128, 126),
                                  (1024, 1024), (136, 100)])
def test_rope_heads_and_parts(dims, interleaved, dtype):
    hd, rot = dims
    check(37, 3, hd, rot, dtype, interleaved, False, far=5000, pad=24)
    check(37, 3, hd, rot, dtype, interleaved, True, far=5000, in_place=True, pad=8)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dims", [(72, 30, 7), (80, 20, 5), (128, 10, 16), (40, 34, 1), (1024, 1022, 2), (2056, 1018, 2),
                                  (8, 2, 300)])
def test_rope_parts_that_end_inside_a_pack(dims, interleaved, dtype):
    """Halves off the 16-byte packs, rotated parts that end inside one, more packs than a
    block has threads, rows of no token's multiple, in and out of place."""
    hd, rot, heads = dims
    check(29, heads, hd, rot, dtype, interleaved, False, far=5000, pad=8, in_place=True)
    check(29, heads, hd, rot, dtype, interleaved, True, far=5000, pad=16)


@pytest.mark.parametrize("T", [1, 2, 63, 1000, 4097])
def test_rope_lengths_and_wrapped_rows(T):
    check(T, 12, 64, 64, BF, False, False, given=False, seq_len=100)
    check(T, 1, 64, 32, F32, True, False, given=False)


@pytest.mark.parametrize("far", [2 ** 21, 2 ** 31 + 12345])
def test_rope_far_positions(far):
    check(200, 2, 64, 64, F32, False, False, far=far)


def test_rope_negative_positions_turn_back():
    """Position -n undoes position n."""
    x = torch.randn(50, 128, device="cuda")
    f = qat.rope_freqs(64)[0]
    pos = torch.randint(0, 100000, (50,), device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    qat.qat_rope(x, y, 2, 64, f, positions=pos)
    qat.qat_rope(y, z, 2, 64, f, positions=-pos)
    torch.cuda.synchronize()
    assert float((z - x).abs().max()) <= 4 * PAIR * 2 * float(x.abs().max())


def test_rope_offsets_past_32_bits():
    """Rows whose element offsets pass 2^31: the last row of a wide, strided tensor."""
    T, ld = 2100, 1 << 20
    x = torch.zeros(T, ld, dtype=BF, device="cuda")
    x[:, :64] = torch.randn(T, 64, device="cuda").to(BF)
    y = torch.empty(T, 64, dtype=BF, device="cuda")
    f = qat.rope_freqs(64)[0]
    qat.qat_rope(x[:, :64], y, 1, 64, f)
    torch.cuda.synchronize()
    ref, mag = rotate(f64(x[:, :64]), 1, 64, f64(f), torch.arange(T), False, 1.0, False)
    within(y, ref, PAIR * mag + U * ref.abs(), "rotated")


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_rope_scaled_contexts(scaling):
    freqs, m = qat.rope_freqs(64, 10000.0, scaling, 8.0, trained_len=1024)
    check(300, 2, 64, 64, F32, False, False, far=8192, scale=m, freqs=freqs)


def test_rope_inverse_is_the_gradient():
    """<R x, y> = <x, R^T y>, and the difference quotient of <R x, y> along a direction."""
    g = torch.Generator().manual_seed(1)
    x, y, d = (torch.randn(40, 160, generator=g).cuda() for _ in range(3))
    f, m = qat.rope_freqs(48, scaling="yarn", factor=4.0, trained_len=512)
    fwd = lambda t: (o := torch.empty_like(t), qat.qat_rope(t, o, 2, 80, f, scale=m))[0]
    back = torch.empty_like(y)
    qat.qat_rope(y, back, 2, 80, f, scale=m, inverse=True)
    quotient = float(((f64(fwd(x + d)) - f64(fwd(x - d))) * f64(y)).sum()) / 2
    direct = float((f64(back) * f64(d)).sum())
    # linear in x: the quotient is exact up to the roundings of both sides
    allowed = 3 * PAIR * m * float(((x.abs() + d.abs()).double().cpu().amax() * 2 * y.abs().double().cpu()).sum())
    assert abs(quotient - direct) <= allowed


def test_rope_stream_and_graph():
    x = torch.randn(100, 128, device="cuda")
    f = qat.rope_freqs(64)[0]
    want, got = torch.empty_like(x), torch.zeros_like(x)
    qat.qat_rope(x, want, 2, 64, f)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        qat.qat_rope(x, got, 2, 64, f)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, got)
    other = torch.zeros_like(x)
    qat.qat_rope(x, other, 2, 64, f, stream=s)
    s.synchronize()
    assert torch.equal(want, other)


def test_rope_refusals():
    x = torch.randn(10, 128, device="cuda")
    y, f = torch.empty_like(x), qat.rope_freqs(64)[0]
    pos = torch.arange(10, device="cuda")

    def bad(code, *a, **k):
        with pytest.raises(qat.QatError) as e:
            qat.qat_rope(*a, **k)
        assert e.value.code == code

    before = qat.launch_count()
    bad(qat.QAT_ERR_ARG, x.half(), y.half(), 2, 64, f)
    bad(qat.QAT_ERR_ARG, x, y.bfloat16(), 2, 64, f)
    bad(qat.QAT_ERR_ARG, x, y[:9], 2, 64, f)
    bad(qat.QAT_ERR_ARG, x, y, 3, 64, f)
    bad(qat.QAT_ERR_ARG, x, y, 2, 64, f.float())
    bad(qat.QAT_ERR_ARG, x, y, 2, 64, f, positions=pos.int())
    bad(qat.QAT_ERR_ARG, x, y, 2, 64, f, positions=pos[:5])
    bad(qat.QAT_ERR_ARG, x.cpu(), y, 2, 64, f)
    bad(qat.QAT_ERR_SHAPE, x, y, 4, 32, f)
    bad(qat.QAT_ERR_SHAPE, x, y, 2, 60, qat.rope_freqs(20)[0])
    bad(qat.QAT_ERR_ALIGN, torch.empty(1284, device="cuda")[1:1281].view(10, 128), y, 2, 64, f)
    assert qat.launch_count() == before
    assert math.isclose(float(f[0]), 1 / (2 * math.pi))
