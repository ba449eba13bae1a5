"""Parameter gradients of long batches of like-signed addends against sums in
64 bits, in launches whose sequences are not cut: a chain of float32 additions
must not grow with the batch.

Tolerance. At most 256 additions in a row are in float32, each off by at most
2^-24 of a running sum that grows to its end: 256 2^-25 = 7.7e-6 (all of one
sign). The addends' own error: a state that remembers one or two tokens and
four factors, ten times 2^-23 = 1.2e-6; the sum over lanes and the result's
rounding, five times 2^-24. Together 9.2e-6, held to 1.2e-5. (One chain over
the sequences here is off by 3e-5 to 6e-4.)"""

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


def scan_reference(T, x, raw, A, b, c, D, gy):
    """Sums over one sequence of constant operands, in 64 bits: gA, gD, gdt_bias (N equal states)."""
    N = 4
    d, sig = math.log1p(math.exp(raw)), 1 / (1 + math.exp(-raw))
    a, h, hs = math.exp(d * A), 0.0, []
    for _ in range(T):
        hs.append(h)
        h = a * h + d * x * b
    gA, gdb, q = [], [], 0.0
    for t in range(T - 1, -1, -1):
        q = gy * c + q
        w = q * a * hs[t]
        gA.append(d * w)
        gdb.append((x * N * q * b + N * A * w) * sig)
        q = a * q
    return math.fsum(gA), T * gy * x, math.fsum(gdb)


@pytest.mark.parametrize("T", [65536, 16400 + 7])
def test_scan(S, T):
    needs(16)
    B, C, N = 296, 4, 4
    v = dict(x=0.3, dt=0.5, A=-1.0, b=0.7, c=0.9, D=0.6, gy=0.1, bias=0.25)
    f = {n: float(np.float32(a)) for n, a in v.items()}
    act = {n: full(v[n], B, T, C) for n in ("x", "dt", "b", "c", "gy")}
    got = S.wkv_scan_backward(act["x"], act["dt"], full(v["A"], C, N), act["b"], act["c"], act["gy"], full(v["D"], C),
                              dt_bias=full(v["bias"], C))
    from rwkv_wkv_linear_mix_b200 import wkv
    assert wkv.lib().wkv_scan_forward_workspace_bytes(B, T, C, N, 1) == 0  # not cut
    gA, gD, gdb = scan_reference(T, f["x"], f["dt"] + f["bias"], f["A"], f["b"], f["c"], f["D"], f["gy"])
    for n, g, w in (("gA", got[2], gA), ("gD", got[5], gD), ("gdt_bias", got[7], gdb)):
        assert off(g, B * w) < TOL, n
