"""How near the selective scan comes to the definition in float32: bounds that
follow from the lengths, and the mean error of a decay.

A decay is off by at most 2^-23 where it is remembered (the exponential's
2^-23.5, an exponent below 1 rounded to 2^-25), so a state by 2^-23 for each
token it remembers: over 48 tokens 5.7e-6, all of one sign. Sums over 16 to 64
states, the gate and one rounding: ten times 2^-24, 6e-7. Outputs are held to
1e-5, gradients, in which the error of a state meets that of the reverse walk,
to 2e-5."""

import numpy as np
import pytest
import torch

from _dev import dev, host64, need_gpu, rel_err
from test_ssm_scan_gpu import NAMES, draw, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    need_gpu()
    from rwkv_wkv_linear_mix_b200 import ssm
    return ssm


@pytest.fixture(scope="module")
def O():
    from oracle import ssm
    return ssm


@pytest.mark.parametrize("B,T,C,N,G", [(2, 48, 64, 16, 1), (2, 33, 72, 8, 1), (1, 40, 96, 32, 3), (1, 48, 32, 64, 2), (2, 17, 24, 12, 1)])
def test_short_sequences(S, O, B, T, C, N, G):
    i = draw("f32", (B, T), C, N, G, seed=N + T)
    pos, kw, ref = operands(i)
    h0, gf = dev(i["h0"]), dev(i["gf"])
    y, last, ckpt = S.wkv_scan_forward(*pos, **kw, init_state=h0, want_ckpt=True)
    ry, rlast = O.scan_forward(**ref, init_state=i["h0"])
    assert rel_err(host64(y), ry) < 1e-5 and rel_err(host64(last), rlast) < 1e-5
    got = S.wkv_scan_backward(*pos, dev(i["gy"]), **kw, init_state=h0, g_final=gf, ckpt=ckpt, want_g_init=True)
    want = O.scan_backward(gy=i["gy32"], init_state=i["h0"], g_final=i["gf"], **ref)
    for n, g in zip(NAMES, got):
        assert rel_err(host64(g), want[n]) < 2e-5, n


@pytest.mark.parametrize("B", [1, 40])  # cut along T, and not
def test_mean_error_of_a_decay(S, O, B):
    """What states that remember 200 to 500 tokens are off by, on average and
    for one token: the exponential is 1.7e-8 low on average for such decays
    (exponents of -0.01 to -0.001), the correction 2.1e-8, and the other
    roundings have no sign, so that 4e-9 are left; held to 1e-8."""
    rng = np.random.Generator(np.random.PCG64(0))
    T, C, N = 3000, 512, 4
    A = -rng.uniform(0.002, 0.005, size=(C, N)).astype(np.float32)
    dt = rng.uniform(0.5, 1.5, size=(1, T, C)).astype(np.float32)
    x, bc = np.ones((1, T, C), np.float32), np.ones((1, T, N), np.float32)
    wide = lambda a: dev(a).expand(B, -1, -1).contiguous()  # noqa: E731
    _, last = S.wkv_scan_forward(wide(x), wide(dt), dev(A), wide(bc), wide(bc), dt_softplus=False)
    _, want = O.scan_forward(x, dt, A, bc, bc, dt_softplus=False)
    off = host64(last[B - 1:]) / want - 1
    assert abs((off * -A).mean()) < 1e-8
