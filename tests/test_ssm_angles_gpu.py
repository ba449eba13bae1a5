"""Angles of the rotation by position, in full float32 precision at every
position it takes: whole numbers p next to a multiple of pi (so that sin p is
tiny and an angle's absolute error shows whole), and offsets up to 2^53.

Frequency 1, so that the angle is p itself, exactly. Tolerance, relative to
each value: the reciprocal root 2, its and the sine's product 1, the sine 1, the
angle's correction 1 and the pair's products 2 units of 2^-23: 8.4e-7, held
to 1e-6."""

import numpy as np
import pytest
import torch

from _dev import need_gpu

pytestmark = pytest.mark.gpu
TOL = 1e-6
# numerators of pi's continued fraction, and numbers without such a place
NEAR = [3, 22, 333, 355, 710, 103993, 104348, 208341, 312689, 833719, 1146408, 80143857, 245850922, 411557987, 2 ** 31 - 1]


@pytest.fixture(scope="module")
def S():
    need_gpu()
    from rwkv_wkv_linear_mix_b200 import ssm
    return ssm


def check(S, positions, offset, T, expect):
    q = torch.zeros(1, T, 16, device="cuda")
    q[..., 0] = 1.0
    f = torch.ones(8, device="cuda")
    out, _ = S.wkv_norm_rotate(q, None, inv_freq=f, positions=positions, pos_offset=offset, head_size=16, eps=0.0)
    p = np.array([float(x) for x in expect])  # exact below 2^53; numpy reduces large angles exactly
    got = out[0].double().cpu().numpy() / 4   # the norm of (1, 0, ..) is 4 at mean square 1/16
    for g, w in ((got[:, 0], np.cos(p)), (got[:, 8], np.sin(p))):
        assert (np.abs(g - w) / np.abs(w)).max() < TOL


@pytest.mark.parametrize("sign", [1, -1])
def test_positions_near_multiples_of_pi(S, sign):
    p = [sign * n for n in NEAR]
    check(S, torch.tensor([p], dtype=torch.int32).cuda(), 0, len(p), p)


@pytest.mark.parametrize("offset", [10 ** 6, 2 ** 32 + 1, 2 ** 40 + 12345, -(2 ** 45) - 7, 2 ** 53 - 64, -(2 ** 53)])
def test_far_offsets(S, offset):
    check(S, None, offset, 64, [offset + t for t in range(64)])


def test_gradient_turns_back_by_the_same_angle(S):
    """With x all ones and eps = 0 the norm's own part of the gradient is known:
    gx = gn - mean(gn), gn the gradient turned back."""
    p = [n for n in NEAR]
    T = len(p)
    x = torch.ones(1, T, 16, device="cuda")
    g = torch.zeros(1, T, 16, device="cuda")
    g[..., 8] = 1.0
    w = torch.ones(16, device="cuda")
    _, _, gw, _ = S.wkv_norm_rotate_backward(x[:, 3:4].contiguous(), None, g[:, 3:4].contiguous(), None, w,
                                             inv_freq=torch.ones(8, device="cuda"),
                                             positions=torch.tensor([p[3:4]], dtype=torch.int32).cuda(), head_size=16, eps=0.0)
    assert abs(gw[0].item() / np.sin(355.0) - 1) < TOL and abs(gw[8].item() / np.cos(355.0) - 1) < TOL


def turned(S, offset, freq):
    q = torch.zeros(1, 64, 16, device="cuda")
    q[..., 0] = 1.0
    out, _ = S.wkv_norm_rotate(q, None, inv_freq=torch.full((8,), freq, device="cuda"), pos_offset=offset, head_size=16, eps=0.0)
    got = out[0].double().cpu().numpy() / 4
    return got[:, 0], got[:, 8]


@pytest.mark.parametrize("offset,freq", [(2 ** 31 + 5, 4096.0), (2 ** 53 - 64, 8.0), (-(2 ** 53), 2.0 ** 12)])
def test_far_offsets_at_high_frequencies(S, offset, freq):
    """Angles of up to 2^65 (whole numbers of 53 bits, so that float64 holds
    them): more turns than float64 counts one by one. 1 / 2 pi in two parts is
    right to 2^-109, so the turns to 2^-44."""
    angle = np.array([float(offset + t) * freq for t in range(64)])
    for g, w in zip(turned(S, offset, freq), (np.cos(angle), np.sin(angle))):
        assert (np.abs(g - w) / np.abs(w)).max() < TOL


def test_a_turn_stays_a_turn(S):
    """At frequencies whose angles no one can know, (1, 0) still goes to a
    point of the unit circle."""
    for freq in (2.0 ** 40, 3e38):
        c, s = turned(S, 2 ** 53 - 64, freq)
        assert np.abs(c * c + s * s - 1).max() < 2 * TOL
