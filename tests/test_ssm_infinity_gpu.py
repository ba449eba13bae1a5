"""How far an infinity reaches in the selective scan: where the definition
gives an infinity the kernels give the same one, where it gives a number they
give that number, whatever states, channels and skip terms there are.

Every operand is positive, so that the infinities of the definition have one
sign. Tolerance of the finite values: a decay off by 3.5e-7 for each of at
most 48 tokens (1.7e-5) and sums of a few 2^-24, held to 3e-5."""

import numpy as np
import pytest

from _dev import dev, host64, need_gpu

pytestmark = pytest.mark.gpu
TOL = 3e-5
INF = float("inf")


@pytest.fixture(scope="module")
def S():
    need_gpu()
    from rwkv_wkv_linear_mix_b200 import ssm
    return ssm


@pytest.fixture(scope="module")
def O():
    from oracle import ssm
    return ssm


def draw(lead, C, N, G, seed, states):
    rng = np.random.Generator(np.random.PCG64(seed))
    i = {n: rng.uniform(0.5, 1.5, size=(*lead, w)).astype(np.float32)
         for n, w in (("x", C), ("dt", C), ("z", C), ("gy", C), ("Bm", G * N), ("Cm", G * N))}
    i["A"] = -rng.uniform(0.2, 1.2, size=(C, N)).astype(np.float32)
    i["D"] = rng.uniform(0.5, 1.5, size=C).astype(np.float32)
    i["dt_bias"] = rng.uniform(-4, -2, size=C).astype(np.float32)
    i["h0"] = rng.uniform(0.1, 0.5, size=(states, C, N)).astype(np.float32)
    return i


def put(i):
    return [dev(i[n]) for n in ("x", "dt", "A", "Bm", "Cm")], dict(D=dev(i["D"]), z=dev(i["z"]), dt_bias=dev(i["dt_bias"]))


def ref(i):
    return {n: i[n] for n in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias")}


def same(got, want, what):
    got = host64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    wild = np.isinf(want)
    assert np.array_equal(np.isinf(got), wild) and np.array_equal(got[wild], want[wild]), what
    fine = np.isfinite(want)
    if fine.any():
        w = want[fine]
        err = np.abs(got[fine] - w) / np.maximum(np.abs(w), max(np.sqrt(np.mean(w * w)), 1e-6))
        assert err.max() < TOL, what


STATES = [4, 12, 16, 24, 40]  # 16 fills its lanes, the others leave some without a state


@pytest.mark.parametrize("N", STATES)
@pytest.mark.parametrize("T", [40, 48])
def test_forward(S, O, N, T):
    i = draw((2, T), 24, N, 1, N, 2)
    i["x"][0, 5, 3] = INF
    pos, kw = put(i)
    y, last = S.wkv_scan_forward(*pos, **kw, init_state=dev(i["h0"]))
    with np.errstate(all="ignore"):
        ry, rlast = O.scan_forward(**ref(i), init_state=i["h0"])
    assert np.isinf(ry).sum() == T - 5
    same(y, ry, "y")
    same(last, rlast, "final state")


@pytest.mark.parametrize("N", STATES)
def test_backward(S, O, N):
    i = draw((2, 48), 24, N, 1, N, 2)
    i["x"][0, 5, 3] = INF
    pos, kw = put(i)
    h0 = dev(i["h0"])
    got = S.wkv_scan_backward(*pos, dev(i["gy"]), **kw, init_state=h0, want_g_init=True)
    with np.errstate(all="ignore"):
        want = O.scan_backward(gy=i["gy"], init_state=i["h0"], **ref(i))
    for n, g in zip(("gx", "gdt", "gA", "gB", "gC", "gD", "gz", "gdt_bias", "g_init"), got):
        same(g, want[n], n)


@pytest.mark.parametrize("N", STATES)
def test_slots_and_single_tokens(S, O, N):
    lengths = [5, 19, 0, 24]
    i = draw((48,), 24, N, 1, N, 4)
    i["x"][8, 3] = INF  # the fourth token of slot 1
    pos, kw = put(i)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    state = dev(i["h0"])
    y = S.wkv_scan_chunk_step(*pos, dev(cu), state, **kw)
    one = {n: a[8:12] if a.shape[0] == 48 else a for n, a in i.items()}
    p1, k1 = put(one)
    state1 = dev(i["h0"])
    y1 = S.wkv_scan_decode_step(*p1, state1, **k1)
    with np.errstate(all="ignore"):
        for s, n in enumerate(lengths):
            if n:
                part = {k: a[None, cu[s]:cu[s + 1]] if a.shape[0] == 48 else a for k, a in ref(i).items()}
                ry, rlast = O.scan_forward(**part, init_state=i["h0"][s:s + 1])
                same(y[cu[s]:cu[s + 1]], ry[0], s)
                same(state[s:s + 1], rlast, s)
        tok = {k: a[:, None] if k not in ("A", "D", "dt_bias") else a for k, a in ref(one).items()}
        ry, rlast = O.scan_forward(**tok, init_state=i["h0"])
    same(y1, ry[:, 0], "single tokens")
    same(state1, rlast, "state")


@pytest.mark.parametrize("gate", [True, False])
def test_without_a_skip_term(S, O, gate):
    """With no D there is no product of it: an infinite x gives an infinite y
    and gz, an infinite gy an infinite gx."""
    i = draw((2, 48), 24, 16, 1, 7, 2)
    i["x"][0, 5, 3] = INF
    i["gy"][1, 20, 8] = INF
    pos, kw = put(i)
    r = ref(i)
    r["D"] = kw["D"] = None
    if not gate:
        r["z"] = kw["z"] = None
    h0 = dev(i["h0"])
    y, _ = S.wkv_scan_forward(*pos, **kw, init_state=h0)
    got = S.wkv_scan_backward(*pos, dev(i["gy"]), **kw, init_state=h0)
    state, one = dev(i["h0"]), [a if a.shape[0] == 24 else a[:, 5].contiguous() for a in pos]
    y1 = S.wkv_scan_decode_step(*one, state, dt_bias=kw["dt_bias"], z=kw["z"][:, 5].contiguous() if gate else None)
    with np.errstate(all="ignore"):
        ry, _ = O.scan_forward(**r, init_state=i["h0"])
        want = O.scan_backward(gy=i["gy"], init_state=i["h0"], **r)
        tok = {k: a if a is None or k in ("A", "dt_bias") else a[:, 5:6] for k, a in r.items()}
        r1, _ = O.scan_forward(**tok, init_state=i["h0"])
    assert np.isinf(ry).any() and np.isinf(want["gx"]).any()
    same(y, ry, "y")
    same(y1, r1[:, 0], "single tokens")
    for n, g in zip(("gx", "gdt", "gA", "gB", "gC", "gD", "gz", "gdt_bias"), got):
        if g is not None:
            same(g, want[n], n)
