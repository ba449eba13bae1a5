"""GPU parity of the per-head norm with position rotation and its backward
against the fp64 oracle.

Tolerances (relative to the value, floored at the rms). float32: the sum of
squares is 8 + 5 additions deep (8e-7, halved by the root), the reciprocal
root 2 ulp, four products, and the rotation's sine and cosine (2^-23 and an
angle rounding of 2^-25 half turns) against pairs of a few rms: below 1e-5;
the backward subtracts two such terms: 2e-5. bf16 adds its one rounding of
2^-8. The weight sums chain at most ~100 additions of partial sums within a
few rms of the result: 2.4e-5, held to 1e-4."""

import numpy as np
import pytest
import torch

from _dev import dev, host64, need_gpu, rel_err
from rwkv_wkv_linear_mix_b200 import synth

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 2.0 ** -8 + 1e-5}
TOL_G = {"f32": 2e-5, "bf16": 2.0 ** -8 + 2e-5}
TOL_SUM = 1e-4


@pytest.fixture(scope="module")
def S():
    need_gpu()
    from rwkv_wkv_linear_mix_b200 import ssm
    return ssm


@pytest.fixture(scope="module")
def O():
    from oracle import ssm
    return ssm


def draw(dtype, seed, **shapes):
    rng = np.random.Generator(np.random.PCG64(seed))
    out = {}
    for n, shape in shapes.items():
        out[n], out[n + "32"] = synth._store(rng.standard_normal(shape, dtype=np.float32), dtype)
    return out, rng


def freqs(R):
    return (10000.0 ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32)


# B, T, Hq, Hk, K, R, interleaved
CASES = [(2, 33, 4, 4, 64, 64, False), (2, 33, 4, 1, 64, 32, False), (1, 1, 1, 0, 8, 8, True), (3, 7, 0, 3, 16, 16, False),
         (1, 50, 5, 2, 80, 48, True), (1, 50, 5, 2, 80, 80, False), (2, 19, 3, 2, 128, 128, False), (1, 65, 2, 2, 256, 256, False),
         (2, 9, 7, 3, 96, 96, True), (1, 300, 1, 1, 24, 16, False), (5, 4, 33, 1, 32, 2, True), (2, 20, 2, 2, 72, 0, False),
         (40, 1, 32, 8, 64, 64, False), (1, 700, 3, 3, 8, 0, False)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hk,K,R,il", CASES)
def test_forward_and_backward_match_oracle(S, O, dtype, B, T, Hq, Hk, K, R, il):
    i, rng = draw(dtype, B + T + K + R, q=(B, T, Hq * K), k=(B, T, Hk * K), gq=(B, T, Hq * K), gk=(B, T, Hk * K))
    wq, wk = rng.uniform(0.5, 1.5, size=(2, K)).astype(np.float32)
    if (B + T) % 3 == 0:
        wk = None
    if (B + T) % 2:
        pos, po, off = rng.integers(-(1 << 31), (1 << 31) - 1, size=(B, T)), True, 0
    else:
        off, po = 1000, False
        pos = np.broadcast_to(off + np.arange(T), (B, T))
    f = freqs(R) if R else None
    put = lambda a: None if a is None else dev(a)  # noqa: E731
    pick = lambda n, H: dev(i[n]) if H else None  # noqa: E731
    q, k, gq, gk = pick("q", Hq), pick("k", Hk), pick("gq", Hq), pick("gk", Hk)
    args = (put(wq), put(wk), put(f), dev(pos.astype(np.int32)) if po else None)
    how = dict(head_size=K, eps=1e-5, pos_offset=off, interleaved=il)
    out = S.wkv_norm_rotate(q, k, *args, **how)
    back = S.wkv_norm_rotate_backward(q, k, gq, gk, *args, **how)
    for j, (n, H, w) in enumerate((("q", Hq, wq), ("k", Hk, wk))):
        if not H:
            assert out[j] is None and back[j] is None
            if w is not None:
                assert not back[2 + j].any()
            continue
        assert rel_err(host64(out[j]), O.norm_rotate(i[n + "32"], w, f, pos, K, 1e-5, il)) < TOL[dtype], n
        rg, rw = O.norm_rotate_backward(i[n + "32"], i["g" + n + "32"], w, f, pos, K, 1e-5, il)
        assert rel_err(host64(back[j]), rg) < TOL_G[dtype], "g" + n
        if w is None:
            assert back[2 + j] is None
        else:
            assert rel_err(host64(back[2 + j]), rw) < TOL_SUM, "gw" + n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_gives_the_same_bits(S, dtype):
    i, rng = draw(dtype, 1, q=(2, 50, 4 * 64), k=(2, 50, 2 * 64), gq=(2, 50, 4 * 64), gk=(2, 50, 2 * 64))
    q, k, gq, gk, f = dev(i["q"]), dev(i["k"]), dev(i["gq"]), dev(i["gk"]), dev(freqs(64))
    qo, ko = S.wkv_norm_rotate(q, k, inv_freq=f, head_size=64)
    a, b, _, _ = S.wkv_norm_rotate_backward(q, k, gq, gk, inv_freq=f, head_size=64)
    S.wkv_norm_rotate_backward(q, k, gq, gk, inv_freq=f, head_size=64, gq=gq, gk=gk)
    assert torch.equal(gq, a) and torch.equal(gk, b)
    S.wkv_norm_rotate(q, k, inv_freq=f, head_size=64, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_rows_of_zeros(S):
    """A head of zeros gives zeros with eps > 0, and finite gradients."""
    q = torch.zeros(1, 3, 2 * 16, device="cuda")
    q[0, 1, :16] = 1.0
    f = dev(freqs(16))
    out, _ = S.wkv_norm_rotate(q, None, inv_freq=f, head_size=16, eps=1e-6)
    assert not out[0, 0].any() and not out[0, 1, 16:].any() and torch.isfinite(out).all()
    g, _, _, _ = S.wkv_norm_rotate_backward(q, None, torch.ones_like(q), None, inv_freq=f, head_size=16, eps=1e-6)
    assert torch.isfinite(g).all()


def test_far_positions_keep_their_angles(S):
    """Position 2^31 - 1 with frequency 1: the angle is known to 64 bits."""
    p = 2 ** 31 - 1
    q = torch.zeros(1, 1, 16, device="cuda")
    q[0, 0, 0] = 1.0
    f = torch.ones(8, device="cuda")
    out, _ = S.wkv_norm_rotate(q, None, inv_freq=f, positions=torch.tensor([[p]], dtype=torch.int32).cuda(), head_size=16,
                               eps=0.0)
    # the norm of (1, 0, ..) is 4 at mean square 1/16
    assert abs(out[0, 0, 0].item() / 4 - np.cos(float(p))) < 1e-6
    assert abs(out[0, 0, 8].item() / 4 - np.sin(float(p))) < 1e-6
    shifted, _ = S.wkv_norm_rotate(q, None, inv_freq=f, pos_offset=p, head_size=16, eps=0.0)
    assert torch.equal(out, shifted)


def test_empty_problems(S):
    none = torch.zeros(2, 0, 64, device="cuda")
    q, k = S.wkv_norm_rotate(none, none, head_size=64)
    assert q.shape == none.shape and k.shape == none.shape
    w = torch.ones(64, device="cuda")
    gq, gk, gwq, gwk = S.wkv_norm_rotate_backward(none, none, none, none, w, w, head_size=64)
    assert not gwq.any() and not gwk.any()


def test_deterministic_whatever_the_workspace_holds(S):
    i, _ = draw("bf16", 4, q=(3, 2000, 256), gq=(3, 2000, 256))
    q, gq, w = dev(i["q"]), dev(i["gq"]), torch.ones(64, device="cuda")
    from rwkv_wkv_linear_mix_b200 import wkv
    need = wkv.lib().wkv_norm_rotate_backward_workspace_bytes(3, 2000, 4, 0, 64)
    runs = []
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        runs.append(S.wkv_norm_rotate_backward(q, None, gq, None, w, inv_freq=dev(freqs(64)), head_size=64, workspace=ws))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][2], runs[1][2])


@pytest.mark.parametrize("K,R,il", [(64, 64, False), (16, 10, True)])
def test_what_shared_memory_held_before_stays_out(S, K, R, il):
    """Tokens past the end of a CTA's share have no angles: what another kernel
    left in shared memory there (NaN, from a scan of NaN) must not reach the
    weight sums."""
    nan = torch.full((8, 64, 4096), float("nan"), device="cuda")
    bc = torch.full((8, 64, 16), float("nan"), device="cuda")
    for _ in range(2):
        S.wkv_scan_backward(nan, nan, nan[0, :1].expand(16, 4096).t().contiguous(), bc, bc, nan)
    q = torch.randn(1, 301, 3 * K, device="cuda")
    w = torch.ones(K, device="cuda")
    gq, _, gw, _ = S.wkv_norm_rotate_backward(q, None, torch.randn_like(q), None, w, inv_freq=dev(freqs(R)), head_size=K,
                                              interleaved=il)
    assert torch.isfinite(gq).all() and torch.isfinite(gw).all()


@pytest.mark.parametrize("il", [False, True])
def test_entries_from_R_on_are_left_as_they_are(S, il):
    """An infinite gradient of an entry that does not turn stays where it is
    (after the norm's own sums: its row), and no other row sees it."""
    K, R = 32, 16
    q = torch.randn(1, 5, 2 * K, device="cuda")
    g = torch.randn(1, 5, 2 * K, device="cuda")
    g[0, 2, R + 3] = float("inf")
    w = torch.ones(K, device="cuda")
    gq, _, gw, _ = S.wkv_norm_rotate_backward(q, None, g, None, w, inv_freq=dev(freqs(R)), head_size=K, interleaved=il)
    bad = torch.zeros(1, 5, 2, dtype=torch.bool, device="cuda")
    bad[0, 2, 0] = True
    assert torch.equal(~torch.isfinite(gq).view(1, 5, 2, K).all(-1), bad)
    fine = torch.ones(K, dtype=torch.bool, device="cuda")
    fine[R + 3] = False
    assert torch.equal(torch.isfinite(gw), fine)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hk,K,R", [(1, 3, 3, 1, 64, 64), (2, 45, 5, 2, 80, 16), (1, 701, 33, 6, 16, 0)])
def test_no_eps(S, O, dtype, B, T, Hq, Hk, K, R):
    """eps = 0 with heads and tokens that leave some lanes without a row: their
    reciprocal root of nothing stays out of the weight sums."""
    i, rng = draw(dtype, T, q=(B, T, Hq * K), k=(B, T, Hk * K), gq=(B, T, Hq * K), gk=(B, T, Hk * K))
    wq, wk = rng.uniform(0.5, 1.5, size=(2, K)).astype(np.float32)
    f, pos = freqs(R) if R else None, np.broadcast_to(np.arange(T), (B, T))
    back = S.wkv_norm_rotate_backward(dev(i["q"]), dev(i["k"]), dev(i["gq"]), dev(i["gk"]), dev(wq), dev(wk),
                                      None if f is None else dev(f), head_size=K, eps=0.0)
    for j, (n, w) in enumerate((("q", wq), ("k", wk))):
        rg, rw = O.norm_rotate_backward(i[n + "32"], i["g" + n + "32"], w, f, pos, K, 0.0, False)
        assert rel_err(host64(back[j]), rg) < TOL_G[dtype], "g" + n
        assert rel_err(host64(back[2 + j]), rw) < TOL_SUM, "gw" + n
