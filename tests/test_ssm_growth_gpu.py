"""A sequence cut along T carries states over its pieces as the uncut walk
does where the product of a piece's decays leaves float32: nothing stays
nothing under unbounded growth, and an infinity stays one under a decay that
comes to zero.

Tolerance: at most 30 growing tokens, each off by 3.5e-7 and by the rounding
of an exponent of 2 log2 e (1.2e-7 log 2): 1.3e-5, held to 3e-5, relative to
each value."""

import numpy as np
import pytest
import torch

from _dev import dev, host64, need_gpu

pytestmark = pytest.mark.gpu
TOL = 3e-5
B, T, C, N, LIVE = 1, 2000, 64, 16, 30


@pytest.fixture(scope="module")
def S():
    need_gpu()
    from rwkv_wkv_linear_mix_b200 import ssm, wkv
    assert wkv.lib().wkv_scan_forward_workspace_bytes(B, T, C, N, 1) > 0  # cut
    return ssm


@pytest.fixture(scope="module")
def O():
    from oracle import ssm
    return ssm


def draw(seed):
    rng = np.random.Generator(np.random.PCG64(seed))
    i = {n: rng.uniform(0.5, 1.5, size=(B, T, w)).astype(np.float32)
         for n, w in (("x", C), ("gy", C), ("Bm", N), ("Cm", N))}
    i["dt"] = np.ones((B, T, C), np.float32)
    i["A"] = rng.uniform(1.5, 2.0, size=(C, N)).astype(np.float32)
    return i


def put(i):
    return [dev(i[n]) for n in ("x", "dt", "A", "Bm", "Cm")], {n: i[n] for n in ("x", "dt", "A", "Bm", "Cm")}


def close(got, want):
    got, on = host64(got), want != 0
    assert np.array_equal(got[~on], want[~on])
    return not on.any() or (np.abs(got[on] - want[on]) / np.abs(want[on])).max() < TOL


def test_growth_after_nothing(S, O):
    """Tokens of zeros, e^3000 of growth, then live tokens."""
    i = draw(0)
    i["x"][:, :-LIVE] = 0
    pos, ref = put(i)
    y, last = S.wkv_scan_forward(*pos, dt_softplus=False)
    ry, rlast = O.scan_forward(**ref, dt_softplus=False)
    assert np.isfinite(ry).all() and close(y, ry) and close(last, rlast)


def test_growth_before_nothing(S, O):
    """The same for the gradients, which are walked down."""
    i = draw(1)
    i["x"][:] = 0
    i["gy"][:, LIVE:] = 0
    pos, ref = put(i)
    got = S.wkv_scan_backward(*pos, dev(i["gy"]), dt_softplus=False, want_g_init=True)
    want = O.scan_backward(gy=i["gy"], dt_softplus=False, **ref)
    assert np.isfinite(want["gx"]).all()
    for k, n in ((0, "gx"), (2, "gA"), (3, "gB"), (4, "gC"), (8, "g_init")):
        assert close(got[k], want[n]), n


def test_growth_of_little(S, O):
    """A state of 1e-36 that grows by e^110 over the sequence: the growth of
    several pieces is past float32 at times, the state never is."""
    i = draw(2)
    i["x"][:], i["A"][:], i["dt"][:] = 0, 1.0, 0
    i["dt"][:, 400:510] = 1.0  # e^80 in one piece of 80 tokens, and more
    h0 = np.full((B, C, N), 1e-36, np.float32)
    pos, ref = put(i)
    y, last = S.wkv_scan_forward(*pos, dt_softplus=False, init_state=dev(h0))
    ry, rlast = O.scan_forward(**ref, init_state=h0, dt_softplus=False)
    assert rlast.max() < 1e13
    # 110 growing tokens
    for g, w in ((y, ry), (last, rlast)):
        assert (np.abs(host64(g) - w) / w).max() < 110 / LIVE * TOL


def test_growth_of_little_in_one_piece(S, O):
    i = draw(3)
    i["x"][:], i["A"][:], i["dt"][:] = 0, 1.0, 0
    i["dt"][:, 410:420] = 11.0  # e^110 within a piece
    h0 = np.full((B, C, N), 1e-36, np.float32)
    pos, ref = put(i)
    y, last = S.wkv_scan_forward(*pos, dt_softplus=False, init_state=dev(h0))
    ry, rlast = O.scan_forward(**ref, init_state=h0, dt_softplus=False)
    for g, w in ((y, ry), (last, rlast)):
        # ten exponents of 16 and their roundings of 2^-21, 4.8e-7 log 2 each; four quarters of the sum of 159
        assert (np.abs(host64(g) - w) / w).max() < TOL


def test_infinity_under_decay(S, O):
    """An infinite token near the start, decays of e^-100 and less over a piece."""
    i = draw(4)
    i["A"], i["dt"] = -i["A"], i["dt"] * np.float32(1.0)
    i["x"][0, 3, 5] = float("inf")
    i["gy"][0, T - 4, 9] = float("inf")
    pos, ref = put(i)
    y, last = S.wkv_scan_forward(*pos, dt_softplus=False)
    gx, *_ = S.wkv_scan_backward(*pos, dev(i["gy"]), dt_softplus=False)
    with np.errstate(all="ignore"):
        ry, rlast = O.scan_forward(**ref, dt_softplus=False)
        want = O.scan_backward(gy=i["gy"], dt_softplus=False, **ref)["gx"]
    for g, w in ((y, ry), (last, rlast), (gx, want)):
        g = host64(g)
        wild = np.isinf(w)
        assert wild.any() and not np.isnan(w).any()
        assert np.array_equal(np.isinf(g), wild) and (g[wild] == w[wild]).all() and np.isfinite(g[~wild]).all()
    assert torch.isfinite(y[..., :5]).all()
