"""Parameter gradients of long batches of like-signed addends against sums in
64 bits, in launches whose sequences are not cut: a chain of float32 additions
must not grow with the batch.

Tolerance. At most 256 additions in a row are in float32, each off by at most
2^-24 of a running sum that grows to its end: 256 2^-25 = 7.7e-6 (all of one
sign). The addends' own error: a state that remembers one or two tokens and
four factors, ten times 2^-23 = 1.2e-6; the sum over lanes and the result's
rounding, five times 2^-24. Together 9.2e-6, held to 1.2e-5. (One chain over
the sequences here is off by 5e-5 to 5e-4.)"""

import math

import numpy as np
import pytest
import torch

from _dev import need_gpu

pytestmark = pytest.mark.gpu
TOL = 1.2e-5


@pytest.fixture(scope="module")
def S():
    need_gpu()
    from rwkv_wkv_linear_mix_b200 import ssm
    yield ssm
    torch.cuda.empty_cache()


def needs(gb):
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


def full(value, *shape, dtype=torch.float32):
    return torch.full(shape, value, device="cuda", dtype=dtype)


def off(got, want):
    return (got.double() / want - 1).abs().max().item()


def test_convolution(S):
    needs(8)
    B, T, C, W = 2368, 32768, 4, 4
    f = lambda v: float(np.float32(v))  # noqa: E731
    x, g = full(0.3, B, T, C), full(0.1, B, T, C)
    _, gw, gb, _ = S.wkv_conv_backward(x, full(0.25, W, C), g, full(0.0, C), silu=False)
    n = torch.tensor([B * (T - (W - 1 - j)) for j in range(W)], dtype=torch.float64, device="cuda")[:, None]
    assert off(gw, n * f(0.3) * f(0.1)) < TOL and off(gb, B * T * f(0.1)) < TOL


@pytest.mark.parametrize("B", [1 << 17, 1 << 20])
def test_convolution_of_many_sequences(S, B):
    """One token each: the sum is over partial rows alone."""
    C, W = 8, 2
    f = lambda v: float(np.float32(v))  # noqa: E731
    x, g = full(0.3, B, 1, C), full(0.1, B, 1, C)
    _, gw, gb, _ = S.wkv_conv_backward(x, full(0.25, W, C), g, full(0.0, C), silu=False)
    assert off(gw[1], B * f(0.3) * f(0.1)) < TOL and off(gb, B * f(0.1)) < TOL and not gw[0].any()


def test_norm(S):
    needs(24)
    H, K, T = 16, 256, 606208
    e, eps = torch.bfloat16, 0.64
    x, g = full(1.0, 1, T, H * K, dtype=e), full(0.1, 1, T, H * K, dtype=e)
    gq, _, gw, _ = S.wkv_norm_rotate_backward(x, None, g, None, full(1.0, K), head_size=K, eps=eps, gq=g)
    want = T * H * float(torch.tensor(0.1, dtype=e)) / math.sqrt(1 + float(np.float32(eps)))
    assert off(gw, want) < TOL
