"""The few-token expert layer at the ends of fp32's range, against the plain 64-bit form within its carried rounding bound: activations
too small for a normal number, and large ones that meet large scales of zero weights."""
import pytest
import torch

from test_gpu_moe_w4a16 import check, layer_of, routing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("low", [-133, -128, -124])
def test_smallest_activations(T, low):
    """Multiples of 2^low against scales of 2^125: the products are of ordinary size."""
    d = layer_of(1, 4, 256, 128, 128, b=1, b_dn=1, scaled=False)
    d["sf_gu"][:] = 252
    X = torch.randint(-7, 8, (T, 256), generator=torch.Generator().manual_seed(T)).double() * 2.0 ** low
    check(X.to(torch.bfloat16), *routing(T, T, 4, 2), d)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("low", [-124, -130, -134])
def test_scaled_activations_below_the_normal_numbers(T, low):
    """x diag(1/s) of 2^low: fp32 holds it to 2^-150, the panel's fp16 to 2^-11 of it."""
    d = layer_of(2, 4, 256, 128, 128, b=1, b_dn=1)
    d["sf_gu"][:] = 252
    d["inv_gu"] *= 2.0 ** -30
    X = torch.randn(T, 256, generator=torch.Generator().manual_seed(T)) * 2.0 ** (low + 30)
    check(X.to(torch.bfloat16), *routing(T, T, 4, 2), d)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("size", [20, 60, 100])
def test_large_activations_of_zero_weights_with_a_large_scale(T, size):
    """2^size times a scale of 2^123 is beyond fp32, but the codes there are zero."""
    d = layer_of(3, 4, 256, 128, 128, b=1, b_dn=1, scaled=False)
    d["sf_gu"][:, :, 1] = 250
    d["wq_gu"][:, :, 16:32] = 0
    X = torch.randn(T, 256, generator=torch.Generator().manual_seed(T))
    X[:, 32:64] *= 2.0 ** size
    check(X.to(torch.bfloat16), *routing(T, T, 4, 2), d)
