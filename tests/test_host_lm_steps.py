"""What the composed steps know without a GPU."""
import pytest
import torch

from quantization_aware_tiny_b200 import steps


def core(d, heads, kv_heads, hd, hidden, attention=True):
    """A core's shapes alone (its operands are made by the library)."""
    c = steps.RecurrentCore.__new__(steps.RecurrentCore)
    c.d, c.H = d, hidden
    c.nqkv = (heads + 2 * kv_heads) * hd
    c.W = tuple(torch.empty(s, device="meta") for s in
                ((c.nqkv, d), (d, heads * hd), (hidden, d), (d, hidden)))
    c.attention = steps.CoreAttention(heads, kv_heads, 16) if attention else None
    return c


@pytest.mark.parametrize("shape", [(160, 4, 2, 40, 320), (160, 2, 1, 64, 320), (128, 8, 8, 32, 512)])
def test_core_flops_are_the_products_of_its_weights(shape):
    """Two operations per weight and token forward; with attention every weight has two
    products backward, also where the heads are wider or narrower than the core."""
    T, R = 24, 3
    c = core(*shape)
    weights = sum(w.shape[0] * w.shape[1] for w in c.W)
    assert c.flops(T, R) == 2.0 * T * R * weights
    assert c.flops_bwd(T, R) == 4.0 * T * R * weights
    d, heads, kv_heads, hd, hidden = shape
    if heads * hd == d:
        c.attention = None  # the core's linears alone: O and Q have gradients, K and V have none
        assert c.flops(T, R) == 2.0 * T * R * weights
        assert c.flops_bwd(T, R) == 4.0 * T * R * (2 * d * d + 2 * d * hidden)
