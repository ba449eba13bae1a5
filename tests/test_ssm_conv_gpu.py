"""GPU parity of the short causal convolution and its backward against the
fp64 oracle, and the bit-for-bit identities its documentation promises.

Tolerances (relative to the value, floored at the rms). float32: W + 1
multiply-adds of partial sums up to ~8 times the result's rms, 2^-24 each
(2.4e-6), and the logistic function's 2^-22 + 2^-23 with an argument rounding
of up to 5e-7: below 1e-5 in all. bf16 adds its one rounding of 2^-8. The
parameter sums chain at most ~100 additions of partial sums within a few rms
of the result: 2.4e-5, held to 1e-4."""

import numpy as np
import pytest
import torch

from _dev import dev, host64, need_gpu, rel_err
from rwkv_wkv_linear_mix_b200 import synth

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 2.0 ** -8 + 1e-5}
TOL_SUM = 1e-4


@pytest.fixture(scope="module")
def S():
    need_gpu()
    from rwkv_wkv_linear_mix_b200 import ssm
    ssm.device_error(reset=True)
    return ssm


@pytest.fixture(scope="module")
def O():
    from oracle import ssm
    return ssm


def draw(dtype, W, C, seed, **shapes):
    """Standard normal activations stored in `dtype` (name and name + "32" as
    stored), weight and bias ~ U(-1, 1)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    out = {"w": rng.uniform(-1, 1, size=(W, C)).astype(np.float32), "b": rng.uniform(-1, 1, size=C).astype(np.float32)}
    for n, shape in shapes.items():
        out[n], out[n + "32"] = synth._store(rng.standard_normal(shape, dtype=np.float32), dtype)
    return out


SHAPES = [(2, 64, 128), (3, 100, 72), (1, 1, 8), (2, 2, 16), (2, 3, 24), (1, 257, 1032), (2, 33, 40), (1, 1000, 520)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,C", SHAPES)
def test_forward_and_backward_match_oracle(S, O, dtype, W, B, T, C):
    i = draw(dtype, W, C, B * 13 + T + C + W, x=(B, T, C), xp=(B, W - 1, C), g=(B, T, C))
    variant = (B + T + W) % 4
    act, with_prev, with_bias = variant != 0, variant % 2 == 0, variant != 3
    x, w, g = dev(i["x"]), dev(i["w"]), dev(i["g"])
    xp = dev(i["xp"]) if with_prev else None
    b = dev(i["b"]) if with_bias else None
    rxp, rb = i["xp32"] if with_prev else None, i["b"] if with_bias else None
    y = S.wkv_conv_forward(x, w, b, xp, silu=act)
    assert rel_err(host64(y), O.conv_forward(i["x32"], i["w"], rb, rxp, act=act)) < TOL[dtype]
    got = S.wkv_conv_backward(x, w, g, b, xp, silu=act, want_gx_prev=True)
    want = O.conv_backward(i["x32"], i["w"], i["g32"], rb, rxp, act=act)
    for n, a, r, tol in zip(("gx", "gweight", "gbias", "gx_prev"), got, want, (TOL[dtype], TOL_SUM, TOL_SUM, TOL[dtype])):
        if a is None:
            assert n == "gbias" and not with_bias
        else:
            assert rel_err(host64(a), r) < tol, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 4])
def test_pieces_give_the_same_bits(S, dtype, W):
    i = draw(dtype, W, 264, 5, x=(3, 300, 264))
    x, w, b = dev(i["x"]), dev(i["w"]), dev(i["b"])
    whole = S.wkv_conv_forward(x, w, b)
    for s in (W - 1, 123, 299):
        first = S.wkv_conv_forward(x[:, :s].contiguous(), w, b)
        second = S.wkv_conv_forward(x[:, s:].contiguous(), w, b, x[:, s - W + 1:s].contiguous())
        assert torch.equal(torch.cat([first, second], 1), whole)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_slots_match_forward_bit_for_bit(S, dtype, W):
    """Ragged slots (empty ones, ones shorter than the window) over two calls
    give the bits of one forward per slot; the state is the last W-1 tokens."""
    C, lengths = 136, [[5, 0, 1, 90, 0, 2], [1, 3, 0, 7, 0, 40]]
    n = [sum(v) for v in lengths]
    i = draw(dtype, W, C, 7, x=(sum(n), C), st=(6, W - 1, C))
    x, w, b, state = dev(i["x"]), dev(i["w"]), dev(i["b"]), dev(i["st"])
    start = state.clone()
    parts, seen = [[] for _ in range(6)], [[] for _ in range(6)]
    at = 0
    for call in range(2):
        cu = torch.tensor([0] + lengths[call]).cumsum(0).to(torch.int32)
        xc = x[at:at + n[call]].contiguous()
        y = S.wkv_conv_chunk_step(xc, w, cu.cuda(), state, b)
        for s in range(6):
            parts[s].append(y[cu[s]:cu[s + 1]])
            seen[s].append(xc[cu[s]:cu[s + 1]])
        at += n[call]
    for s in range(6):
        tokens = torch.cat(seen[s])
        if len(tokens):
            want = S.wkv_conv_forward(tokens[None].contiguous(), w, b, start[s:s + 1].contiguous())[0]
            assert torch.equal(torch.cat(parts[s]), want), s
        assert torch.equal(state[s], torch.cat([start[s], tokens])[-(W - 1):]), s
    assert S.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_short_slots_among_long_ones(S, dtype, W):
    """Slots of a few tokens in a batch whose mean length is hundreds: the bits
    of one forward per slot, call after call."""
    C, lengths = 72, [700, 1, 2, 900, 3, 4, 5, 0, 6, 7, 1500, 8, 9, 17]
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    n, slots = int(cu[-1]), len(lengths)
    i = draw(dtype, W, C, 21, x=(n, C), st=(slots, W - 1, C))
    x, w, b, start = dev(i["x"]), dev(i["w"]), dev(i["b"]), dev(i["st"])
    want, after = torch.empty_like(x), start.clone()
    for s, m in enumerate(lengths):
        if m:
            piece = x[cu[s]:cu[s + 1]]
            want[cu[s]:cu[s + 1]] = S.wkv_conv_forward(piece[None].contiguous(), w, b, start[s:s + 1].contiguous())[0]
            after[s] = torch.cat([start[s], piece])[-(W - 1):]
    for _ in range(20):
        state = start.clone()
        y = S.wkv_conv_chunk_step(x, w, cu.cuda(), state, b)
        assert torch.equal(y, want) and torch.equal(state, after)
    assert S.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("slots", [1, 37])
def test_decode_matches_slots_bit_for_bit(S, dtype, W, slots):
    C = 264
    i = draw(dtype, W, C, 9, x=(slots, C), st=(slots, W - 1, C))
    x, w = dev(i["x"]), dev(i["w"])
    a, b = dev(i["st"]), dev(i["st"])
    ya = S.wkv_conv_decode_step(x, w, a, silu=False)
    yb = S.wkv_conv_chunk_step(x, w, torch.arange(slots + 1, dtype=torch.int32).cuda(), b, silu=False)
    assert torch.equal(ya, yb) and torch.equal(a, b)


def test_bad_slots_are_skipped_and_rows_outside_left_alone(S):
    C, W = 64, 4
    x, w = torch.randn(10, C, device="cuda"), torch.randn(W, C, device="cuda")
    state = torch.randn(4, W - 1, C, device="cuda")
    before, y = state.clone(), torch.full_like(x, 7.0)
    # slot 0 decreases, slot 1 starts below 0, slot 2 is fine, slot 3 ends past the tokens
    S.wkv_conv_chunk_step(x, w, torch.tensor([2, -1, 3, 6, 11], dtype=torch.int32).cuda(), state, y=y)
    assert S.device_error() == 2
    want = S.wkv_conv_forward(x[None, 3:6].contiguous(), w, None, before[2:3].contiguous())[0]
    assert torch.equal(y[3:6], want)
    assert (y[:3] == 7).all() and (y[6:] == 7).all()
    keep = torch.tensor([0, 1, 3], device="cuda")
    assert torch.equal(state[keep], before[keep]) and torch.equal(state[2], x[3:6])


def test_empty_problems(S):
    w = torch.randn(4, 16, device="cuda")
    x = torch.zeros(2, 0, 16, device="cuda")
    assert S.wkv_conv_forward(x, w).shape == x.shape
    gx, gw, gb, gp = S.wkv_conv_backward(x, w, x, torch.zeros(16, device="cuda"), want_gx_prev=True)
    assert gx.shape == x.shape and not gw.any() and not gb.any() and not gp.any() and gp.shape == (2, 3, 16)
    state = torch.randn(3, 3, 16, device="cuda")
    before = state.clone()
    none = torch.zeros(0, 16, device="cuda")
    assert S.wkv_conv_chunk_step(none, w, torch.zeros(4, dtype=torch.int32, device="cuda"), state).shape == (0, 16)
    assert torch.equal(state, before) and S.device_error() == 0


def test_infinities_stay_in_their_window(S):
    """A token of inf or NaN reaches the W outputs that see it, and no other."""
    x = torch.randn(1, 40, 8, device="cuda")
    x[0, 20, 3] = float("inf")
    x[0, 5, 1] = float("nan")
    w = torch.rand(4, 8, device="cuda") + 0.1
    y = S.wkv_conv_forward(x, w)
    bad = ~torch.isfinite(y[0])
    want = torch.zeros_like(bad)
    want[20:24, 3] = True
    want[5:9, 1] = True
    assert torch.equal(bad, want)


def test_deterministic_whatever_the_workspace_holds(S):
    i = draw("bf16", 4, 512, 3, x=(4, 700, 512), g=(4, 700, 512))
    x, w, g, b = dev(i["x"]), dev(i["w"]), dev(i["g"]), dev(i["b"])
    from rwkv_wkv_linear_mix_b200 import wkv
    need = wkv.lib().wkv_conv_backward_workspace_bytes(4, 700, 512, 1, 4)
    runs = []
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        runs.append(S.wkv_conv_backward(x, w, g, b, workspace=ws)[:3])
    assert all(torch.equal(p, q) for p, q in zip(*runs))
