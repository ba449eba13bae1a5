"""Pins of the fp64 oracle of the state-space operators (oracle/ssm.py):
hand-worked values, limits with a closed form, and central differences of the
loss in every operand."""

import numpy as np
import pytest

from _pins import rel_err


@pytest.fixture(scope="module")
def S():
    from oracle import ssm
    return ssm


def differences(loss, arrays, name, h=1e-6):
    """Central differences of loss(**arrays) in every entry of arrays[name]."""
    a = arrays[name]
    out = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        up, down = a.copy(), a.copy()
        up[i] += h
        down[i] -= h
        out[i] = (loss(**{**arrays, name: up}) - loss(**{**arrays, name: down})) / (2 * h)
    return out


# ---- convolution --------------------------------------------------------------------------

def test_conv_hand_worked(S):
    """One channel, x = 1, 2, 3, taps (oldest first) 10, 1, bias 0.5: without
    activation 1.5, 2 + 10 + 0.5, 3 + 20 + 0.5; with x_prev = 4 the first
    gets 40 more."""
    x = np.array([1.0, 2, 3]).reshape(1, 3, 1)
    w = np.array([[10.0], [1.0]])
    y = S.conv_forward(x, w, np.array([0.5]), act=False)
    assert np.array_equal(y.ravel(), [1.5, 12.5, 23.5])
    y = S.conv_forward(x, w, np.array([0.5]), x_prev=np.full((1, 1, 1), 4.0), act=False)
    assert np.array_equal(y.ravel(), [41.5, 12.5, 23.5])
    assert abs(S.silu(np.array(2.0)) - 2 / (1 + np.exp(-2.0))) < 1e-15


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", [True, False])
def test_conv_backward_matches_differences(S, W, act):
    rng = np.random.default_rng(W)
    B, T, C = 2, 5, 3
    a = dict(x=rng.normal(size=(B, T, C)), weight=rng.normal(size=(W, C)), bias=rng.normal(size=C),
             x_prev=rng.normal(size=(B, W - 1, C)))
    gy = rng.normal(size=(B, T, C))
    loss = lambda **k: float((gy * S.conv_forward(act=act, **k)).sum())  # noqa: E731
    got = S.conv_backward(a["x"], a["weight"], gy, a["bias"], a["x_prev"], act=act)
    for name, g in zip(("x", "weight", "bias", "x_prev"), got):
        assert rel_err(g, differences(loss, a, name)) < 1e-8, name


# ---- norm and rotation ----------------------------------------------------------------------

def test_norm_rotate_hand_worked(S):
    """x = (3, 4, 0, 0) has mean square 6.25: v = (1.2, 1.6, 0, 0). A quarter
    turn sends the pair (v0, v2) of the split form to (0, 1.2) and the pair
    (v0, v1) of the interleaved form to (-1.6, 1.2)."""
    x = np.array([3.0, 4, 0, 0]).reshape(1, 1, 4)
    f = np.array([np.pi / 2, 0.0])
    pos = np.ones((1, 1))
    y = S.norm_rotate(x, None, f, pos, 4, 0.0, False).ravel()
    assert np.allclose(y, [0, 1.6, 1.2, 0], atol=1e-15)
    y = S.norm_rotate(x, None, f, pos, 4, 0.0, True).ravel()
    assert np.allclose(y, [-1.6, 1.2, 0, 0], atol=1e-15)


def test_rotation_keeps_products_of_equal_distance(S):
    """The product of a query at p and a key at s depends on p - s alone."""
    rng = np.random.default_rng(0)
    K, R = 8, 8
    f = 100.0 ** (-np.arange(0, R, 2) / R)
    q, k = rng.normal(size=(2, 1, 1, K))
    at = lambda v, p: S.norm_rotate(v, None, f, np.full((1, 1), p), K, 1e-6, False).ravel()  # noqa: E731
    assert abs(at(q, 7) @ at(k, 3) - at(q, 1007) @ at(k, 1003)) < 1e-10


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R", [0, 2, 4, 6])
def test_norm_rotate_backward_matches_differences(S, R, interleaved):
    rng = np.random.default_rng(R)
    B, T, H, K, eps = 2, 3, 2, 6, 1e-2
    f = rng.uniform(0.1, 2, size=R // 2) if R else None
    pos = rng.integers(0, 50, size=(B, T))
    a = dict(x=rng.normal(size=(B, T, H * K)), weight=rng.normal(size=K))
    g = rng.normal(size=(B, T, H * K))
    loss = lambda x, weight: float((g * S.norm_rotate(x, weight, f, pos, K, eps, interleaved)).sum())  # noqa: E731
    gx, gw = S.norm_rotate_backward(a["x"], g, a["weight"], f, pos, K, eps, interleaved)
    assert rel_err(gx, differences(loss, a, "x")) < 1e-7
    assert rel_err(gw, differences(loss, a, "weight")) < 1e-7


# ---- scan -------------------------------------------------------------------------------------

def scan_operands(rng, B=2, T=4, C=4, N=3, G=2):
    return dict(x=rng.normal(size=(B, T, C)), dt=rng.normal(size=(B, T, C)), A=-rng.uniform(0.2, 2, size=(C, N)),
                Bm=rng.normal(size=(B, T, G * N)), Cm=rng.normal(size=(B, T, G * N)), D=rng.normal(size=C),
                z=rng.normal(size=(B, T, C)), dt_bias=rng.normal(size=C), init_state=rng.normal(size=(B, C, N)))


def test_scan_matches_the_unrolled_sum(S):
    """h_T = sum_s e^{A (d_{s+1} + .. + d_T)} d_s x_s B_s + e^{A sum d} h_0, summed directly."""
    rng = np.random.default_rng(1)
    o = scan_operands(rng)
    y, h = S.scan_forward(**o)
    d = np.log1p(np.exp(o["dt"] + o["dt_bias"]))
    B, T, C = d.shape
    N = o["A"].shape[1]
    want, wy = np.zeros((B, C, N)), np.zeros((B, T, C))
    for b, c, n in np.ndindex(B, C, N):
        g = c // (C // 2)
        for t in range(T):
            v = np.exp(o["A"][c, n] * d[b, :t + 1, c].sum()) * o["init_state"][b, c, n]
            for s in range(t + 1):
                v += (np.exp(o["A"][c, n] * d[b, s + 1:t + 1, c].sum()) * d[b, s, c] * o["x"][b, s, c] *
                      o["Bm"][b, s, g * N + n])
            wy[b, t, c] += v * o["Cm"][b, t, g * N + n]
        want[b, c, n] = v
    z = o["z"]
    wy = (wy + o["D"] * o["x"]) * z / (1 + np.exp(-z))
    assert rel_err(h, want) < 1e-12 and rel_err(y, wy) < 1e-12


def test_scan_limits(S):
    """A = 0: the state is the running sum of d x B. A very negative: only the
    present token is left, y = (d B.C + D) x."""
    rng = np.random.default_rng(2)
    o = {**scan_operands(rng), "z": None, "init_state": None, "dt_bias": None}
    o["dt"] = rng.uniform(0.1, 1, size=o["dt"].shape)
    _, h = S.scan_forward(**{**o, "A": 0 * o["A"]}, dt_softplus=False)
    Bw = np.repeat(o["Bm"].reshape(2, 4, 2, 3), 2, axis=2)
    assert rel_err(h, ((o["dt"] * o["x"])[..., None] * Bw).sum(1)) < 1e-13
    y, _ = S.scan_forward(**{**o, "A": 0 * o["A"] - 1e4}, dt_softplus=False)
    Cw = np.repeat(o["Cm"].reshape(2, 4, 2, 3), 2, axis=2)
    assert rel_err(y, o["x"] * (o["dt"] * (Bw * Cw).sum(-1) + o["D"])) < 1e-13


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("gate", [True, False])
def test_scan_backward_matches_differences(S, gate, softplus):
    rng = np.random.default_rng(3)
    o = scan_operands(rng)
    if not gate:
        o["z"] = None
    gy, gf = rng.normal(size=o["x"].shape), rng.normal(size=o["init_state"].shape)

    def loss(**k):
        y, h = S.scan_forward(**k, dt_softplus=softplus)
        return float((gy * y).sum() + (gf * h).sum())

    got = S.scan_backward(gy=gy, g_final=gf, dt_softplus=softplus, **o)
    names = dict(x="gx", dt="gdt", A="gA", Bm="gB", Cm="gC", D="gD", z="gz", dt_bias="gdt_bias", init_state="g_init")
    # Rounding of the differences: the loss is a sum of terms of total size M
    # (large without the softplus: negative steps let the state grow), each
    # known to some 16 roundings of 2^-53, and two losses are divided by 2 h.
    y, last = S.scan_forward(**o, dt_softplus=softplus)
    M, h = float(np.abs(gy * y).sum() + np.abs(gf * last).sum()), 1e-6
    for name, g in names.items():
        if o[name] is not None:
            ref = differences(loss, o, name, h)
            tol = 1e-7 + 16 * 2.0 ** -53 * M / h / np.sqrt((ref ** 2).mean())
            assert rel_err(got[g], ref) < tol, name
