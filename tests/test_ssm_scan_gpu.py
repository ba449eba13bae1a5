"""GPU parity of the selective scan (forward, backward, slots, single tokens)
against the fp64 oracle, and the identities its documentation promises.

Tolerances (relative to the value, floored at the rms). A state multiplies by
decays each off by some 3.5e-7 (2^-22 of the exponential, the roundings of
its argument and of the product) for as many tokens as it remembers: at most
300 here, 1.05e-4; with the outputs' own sums of a few 2^-24 that is held to
1.2e-4 for float32, and bf16 outputs add their one rounding of 2^-8. The
gradients of the parameters add up such terms in short chains (a tile, then
a piece, then the rows): the same bound. A state remembers at most
1 / (min d min |A|) = 1 / (0.001 0.6) tokens in the long test: 6e-4."""

import numpy as np
import pytest
import torch

from _dev import dev, host64, need_gpu, rel_err
from rwkv_wkv_linear_mix_b200 import synth

pytestmark = pytest.mark.gpu

TOL32 = 1.2e-4
TOL = {"f32": TOL32, "bf16": 2.0 ** -8 + TOL32}
NAMES = ("gx", "gdt", "gA", "gB", "gC", "gD", "gz", "gdt_bias", "g_init")


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


def draw(dtype, lead, C, N, G, seed, states=None):
    """Operands: `i[n]` as stored, `i[n + "32"]` the stored values. Step sizes
    through the softplus 0.001 .. 0.1 (times e^{N(0, 1/4)}), rates about 1 .. N."""
    rng = np.random.Generator(np.random.PCG64(seed))
    i = {}
    for n, w, std in (("x", C, 1), ("dt", C, 0.5), ("z", C, 1), ("gy", C, 1), ("Bm", G * N, 1), ("Cm", G * N, 1)):
        i[n], i[n + "32"] = synth._store((std * rng.standard_normal((*lead, w))).astype(np.float32), dtype)
    i["A"] = (-np.arange(1, N + 1) * np.exp(0.2 * rng.standard_normal((C, N)))).astype(np.float32)
    i["D"] = rng.uniform(0.5, 1.5, size=C).astype(np.float32)
    i["dt_bias"] = np.log(np.expm1(np.exp(rng.uniform(np.log(1e-3), np.log(0.1), size=C)))).astype(np.float32)
    for n in ("h0", "gf"):
        i[n] = (0.3 * rng.standard_normal((states or lead[0], C, N))).astype(np.float32)
    return i


def operands(i, z=True, D=True, bias=True):
    """(positional and keyword operands on the device, the same for the oracle)"""
    pos = [dev(i[n]) for n in ("x", "dt", "A", "Bm", "Cm")]
    kw = dict(D=dev(i["D"]) if D else None, z=dev(i["z"]) if z else None, dt_bias=dev(i["dt_bias"]) if bias else None)
    ref = dict(x=i["x32"], dt=i["dt32"], A=i["A"], Bm=i["Bm32"], Cm=i["Cm32"], D=i["D"] if D else None,
               z=i["z32"] if z else None, dt_bias=i["dt_bias"] if bias else None)
    return pos, kw, ref


# B, T, C, N, G: all lane counts, padded states, tails of channels and tokens,
# cut along T (long, with few channels) and not
CASES = [(2, 64, 64, 16, 1), (1, 1, 8, 16, 1), (2, 15, 72, 16, 1), (1, 16, 64, 8, 1), (2, 17, 136, 4, 1), (1, 33, 48, 12, 2),
         (2, 40, 96, 32, 3), (1, 47, 56, 24, 1), (1, 50, 32, 64, 2), (2, 31, 24, 40, 1), (1, 300, 64, 16, 1),
         (2, 257, 72, 16, 1), (1, 200, 16, 64, 1), (1, 190, 80, 32, 1), (3, 129, 128, 8, 2), (1, 128, 8, 4, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,N,G", CASES)
def test_forward_and_backward_match_oracle(S, O, dtype, B, T, C, N, G):
    i = draw(dtype, (B, T), C, N, G, seed=B + T + C + N)
    v = (T + N // 4) % 4
    pos, kw, ref = operands(i, z=v != 1, D=v != 2, bias=v != 3)
    h0, gf = (dev(i["h0"]), dev(i["gf"])) if v % 2 == 0 else (None, None)
    rh0, rgf = (i["h0"], i["gf"]) if v % 2 == 0 else (None, None)
    y, last, ckpt = S.wkv_scan_forward(*pos, **kw, init_state=h0, want_ckpt=True)
    ry, rlast, every, _, _ = O.scan_forward(**ref, init_state=rh0, states=True)
    assert rel_err(host64(y), ry) < TOL[dtype]
    assert rel_err(host64(last), rlast) < TOL32
    first = np.zeros((B, C, N)) if rh0 is None else rh0
    want = np.stack([every[:, 16 * m - 1] if m else first for m in range(ckpt.shape[1])], 1)
    assert rel_err(host64(ckpt), want) < TOL32
    want = O.scan_backward(gy=i["gy32"], init_state=rh0, g_final=rgf, **ref)
    for ck in (ckpt, None):
        got = S.wkv_scan_backward(*pos, dev(i["gy"]), **kw, init_state=h0, g_final=gf, ckpt=ck, want_g_init=True)
        for n, g in zip(NAMES, got):
            if g is None:
                assert kw.get(n[1:], 0) is None, n
                continue
            tol = TOL32 if g.dtype == torch.float32 else TOL["bf16"]
            assert rel_err(host64(g), want[n]) < tol, (n, ck is not None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_the_softplus(S, O, dtype):
    i = draw(dtype, (2, 50), 64, 16, 1, seed=3)
    i["dt32"] = np.abs(i["dt32"])
    i["dt"] = synth._store(i["dt32"], dtype)[0]
    pos, kw, ref = operands(i, bias=False)
    y, last = S.wkv_scan_forward(*pos, **kw, dt_softplus=False)
    ry, rlast = O.scan_forward(**ref, dt_softplus=False)
    assert rel_err(host64(y), ry) < TOL[dtype] and rel_err(host64(last), rlast) < TOL32
    got = S.wkv_scan_backward(*pos, dev(i["gy"]), **kw, dt_softplus=False)
    want = O.scan_backward(gy=i["gy32"], dt_softplus=False, **ref)
    for n, g in zip(NAMES, got):
        if g is not None:
            assert rel_err(host64(g), want[n]) < (TOL32 if g.dtype == torch.float32 else TOL[dtype]), n


def test_step_sizes_from_nothing_to_all(S, O):
    """Raw step sizes from -60 (softplus 1e-26) to 60, decays down to e^-1000: no
    overflow, and softplus keeps its relative precision at both ends."""
    i = draw("f32", (1, 40), 16, 16, 1, seed=4)
    i["dt"] = i["dt32"] = np.linspace(-60, 60, 40 * 16).reshape(1, 40, 16).astype(np.float32)
    pos, kw, ref = operands(i, bias=False)
    y, last = S.wkv_scan_forward(*pos, **kw)
    ry, rlast = O.scan_forward(**ref)
    assert rel_err(host64(y), ry) < TOL32 and rel_err(host64(last), rlast) < TOL32
    got = S.wkv_scan_backward(*pos, dev(i["gy"]), **kw)
    want = O.scan_backward(gy=i["gy32"], **ref)
    for n, g in zip(NAMES, got):
        if g is not None:
            assert rel_err(host64(g), want[n]) < TOL32, n


@pytest.mark.parametrize("C,N", [(64, 16), (1024, 16)])
def test_long_sequence(S, O, C, N):
    """8191 tokens in one sequence, cut along T; 4 channels against the oracle
    (channels are independent)."""
    i = draw("f32", (1, 8191), C, N, 1, seed=6)
    pos, kw, ref = operands(i)
    y, last, ckpt = S.wkv_scan_forward(*pos, **kw, want_ckpt=True)
    gx, gdt, gA, _, _, gD, gz, gdb, _ = S.wkv_scan_backward(*pos, dev(i["gy"]), **kw, ckpt=ckpt)
    cs = [0, 1, C // 2 + 1, C - 1]
    ref = {n: a if n in ("Bm", "Cm") else a[..., cs] if n != "A" else a[cs] for n, a in ref.items()}
    ry, rlast = O.scan_forward(**ref)
    assert rel_err(host64(y)[..., cs], ry) < 6e-4 and rel_err(host64(last)[:, cs], rlast) < 6e-4
    want = O.scan_backward(gy=i["gy32"][..., cs], **ref)
    for n, g in (("gx", gx), ("gdt", gdt), ("gz", gz)):
        assert rel_err(host64(g)[..., cs], want[n]) < 6e-4, n
    for n, g in (("gA", gA), ("gD", gD), ("gdt_bias", gdb)):
        assert rel_err(host64(g)[cs], want[n]) < 6e-4, n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_slots_match_forward_bit_for_bit(S, dtype, N):
    """Ragged slots over three calls give the bits of one call, and of an
    uncut forward of each slot."""
    C, G = 80, 1
    lengths = [[5, 0, 1, 90, 0, 2], [1, 17, 0, 3, 0, 40], [0, 16, 0, 32, 0, 1]]
    total = [sum(v[s] for v in lengths) for s in range(6)]
    i = draw(dtype, (sum(total),), C, N, G, seed=8, states=6)
    whole, kw, _ = operands(i)
    cu_all = np.concatenate([[0], np.cumsum(total)]).astype(np.int32)
    st = dev(i["h0"])
    y_all = S.wkv_scan_chunk_step(*whole, dev(cu_all), st, **kw)
    st2 = dev(i["h0"])
    done = [0] * 6
    for call in lengths:
        idx = np.concatenate([np.arange(cu_all[s] + done[s], cu_all[s] + done[s] + call[s]) for s in range(6)])
        it = torch.from_numpy(idx).long().cuda()
        part = [t if n == 2 else t[it].contiguous() for n, t in enumerate(whole)]
        kwp = {**kw, "z": kw["z"][it].contiguous()}
        cu = dev(np.concatenate([[0], np.cumsum(call)]).astype(np.int32))
        y = S.wkv_scan_chunk_step(*part, cu, st2, **kwp)
        assert torch.equal(y, y_all[it])
        done = [a + b for a, b in zip(done, call)]
    assert torch.equal(st, st2)
    from rwkv_wkv_linear_mix_b200 import wkv
    uncut = 0
    for s in range(6):
        a, b = int(cu_all[s]), int(cu_all[s + 1])
        one = [t if n == 2 else t[None, a:b].contiguous() for n, t in enumerate(whole)]
        if b > a and wkv.lib().wkv_scan_forward_workspace_bytes(1, b - a, C, N, G) == 0:
            uncut += 1
            y, last = S.wkv_scan_forward(*one, D=kw["D"], z=kw["z"][None, a:b].contiguous(), dt_bias=kw["dt_bias"],
                                         init_state=dev(i["h0"][s:s + 1]))
            assert torch.equal(y[0], y_all[a:b]) and torch.equal(last[0], st[s])
    assert uncut >= 3 and S.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,G,C", [(4, 1, 64), (8, 2, 48), (16, 1, 136), (16, 3, 72), (24, 1, 64), (32, 1, 40), (64, 2, 48)])
@pytest.mark.parametrize("gate", [True, False])
def test_decode_matches_slots_bit_for_bit(S, O, dtype, N, G, C, gate):
    slots = 5
    i = draw(dtype, (slots,), C, N, G, seed=N + C, states=slots)
    pos, kw, ref = operands(i, z=gate, D=gate, bias=gate)
    a, b = dev(i["h0"]), dev(i["h0"])
    ya = S.wkv_scan_decode_step(*pos, a, **kw)
    yb = S.wkv_scan_chunk_step(*pos, torch.arange(slots + 1, dtype=torch.int32).cuda(), b, **kw)
    assert torch.equal(ya, yb) and torch.equal(a, b)
    tok = {n: v if v is None or n in ("A", "D", "dt_bias") else v[:, None] for n, v in ref.items()}
    ry, rlast = O.scan_forward(**tok, init_state=i["h0"])
    assert rel_err(host64(ya), ry[:, 0]) < TOL[dtype] and rel_err(host64(a), rlast) < TOL32


def test_bad_slots_are_skipped_and_rows_outside_left_alone(S):
    i = draw("f32", (10,), 64, 16, 1, seed=2, states=4)
    pos, kw, _ = operands(i)
    state, y = dev(i["h0"]), torch.full((10, 64), 7.0, device="cuda")
    before = state.clone()
    S.wkv_scan_chunk_step(*pos, torch.tensor([2, -1, 3, 6, 11], dtype=torch.int32).cuda(), state, **kw, y=y)
    assert S.device_error() == 2
    assert (y[:3] == 7).all() and (y[6:] == 7).all() and not (y[3:6] == 7).any()
    keep = torch.tensor([0, 1, 3], device="cuda")
    assert torch.equal(state[keep], before[keep]) and not torch.equal(state[2], before[2])


def test_empty_problems(S):
    i = draw("f32", (2, 0), 16, 8, 1, seed=1)
    pos, kw, _ = operands(i)
    h0, gf = dev(i["h0"]), dev(i["gf"])
    y, last = S.wkv_scan_forward(*pos, **kw, init_state=h0)
    assert y.shape == (2, 0, 16) and torch.equal(last, h0)
    assert not S.wkv_scan_forward(*pos, **kw)[1].any()
    got = S.wkv_scan_backward(*pos, dev(i["gy"]), **kw, g_final=gf, want_g_init=True)
    assert torch.equal(got[8], gf) and not got[2].any() and not got[5].any() and not got[7].any()
    state = dev(i["h0"])
    none = draw("f32", (0,), 16, 8, 1, seed=1, states=2)
    pos, kw, _ = operands(none)
    assert S.wkv_scan_chunk_step(*pos, torch.zeros(3, dtype=torch.int32, device="cuda"), state, **kw).shape == (0, 16)
    assert torch.equal(state, h0) and S.device_error() == 0


def test_state_in_place_and_pieces(S):
    """final_state = init_state works in place, and feeding a batch in two
    uncut pieces gives the bits of one."""
    i = draw("bf16", (2, 100), 64, 16, 1, seed=9)
    pos, kw, _ = operands(i)
    y, last = S.wkv_scan_forward(*pos, **kw, init_state=dev(i["h0"]))
    state, parts = dev(i["h0"]), []
    for a, b in ((0, 37), (37, 100)):
        cut = [t if n == 2 else t[:, a:b].contiguous() for n, t in enumerate(pos)]
        p, _ = S.wkv_scan_forward(*cut, D=kw["D"], z=kw["z"][:, a:b].contiguous(), dt_bias=kw["dt_bias"], init_state=state,
                                  final_state=state)
        parts.append(p)
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(state, last)


@pytest.mark.parametrize("B,T,C", [(1, 2000, 64), (3, 400, 72)])
def test_state_in_place_of_a_cut_launch(S, B, T, C):
    """final_state = init_state where the sequence is cut along T: every piece
    reads the initial state, whatever piece is done first."""
    i = draw("f32", (B, T), C, 16, 1, seed=10)
    pos, kw, _ = operands(i)
    from rwkv_wkv_linear_mix_b200 import wkv
    assert wkv.lib().wkv_scan_forward_workspace_bytes(B, T, C, 16, 1) > 0
    y, last = S.wkv_scan_forward(*pos, **kw, init_state=dev(i["h0"]))
    for _ in range(5):
        state = dev(i["h0"])
        y2, last2 = S.wkv_scan_forward(*pos, **kw, init_state=state, final_state=state)
        assert last2 is state and torch.equal(y2, y) and torch.equal(state, last)


@pytest.mark.parametrize("B,T,C", [(1, 400, 64), (4, 90, 512)])
def test_deterministic_whatever_the_buffers_hold(S, B, T, C):
    i = draw("bf16", (B, T), C, 16, 1, seed=5)
    pos, kw, _ = operands(i)
    from rwkv_wkv_linear_mix_b200 import wkv
    L, runs = wkv.lib(), []
    for fill in (0, 255):
        ws = torch.full((max(16, L.wkv_scan_forward_workspace_bytes(B, T, C, 16, 1)),), fill, dtype=torch.uint8, device="cuda")
        f = S.wkv_scan_forward(*pos, **kw, workspace=ws)
        ws = torch.full((L.wkv_scan_backward_workspace_bytes(B, T, C, 16, 1, 0),), fill, dtype=torch.uint8, device="cuda")
        g = S.wkv_scan_backward(*pos, dev(i["gy"]), **kw, want_g_init=True, workspace=ws)
        runs.append((*f, *g))
    assert all(torch.equal(p, q) for p, q in zip(*runs))


def test_backward_on_a_side_stream_and_in_a_graph(S):
    """The calls go to the current stream, allocate nothing themselves and can
    be captured; a replay on new inputs gives the eager results."""
    i, j = (draw("bf16", (1, 300), 64, 16, 1, seed=s) for s in (11, 12))
    pos, kw, _ = operands(i)
    gy = dev(i["gy"])
    eager = [t for t in (*S.wkv_scan_forward(*pos, **kw), *S.wkv_scan_backward(*pos, gy, **kw)) if t is not None]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [t for t in (*S.wkv_scan_forward(*pos, **kw), *S.wkv_scan_backward(*pos, gy, **kw)) if t is not None]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [t for t in (*S.wkv_scan_forward(*pos, **kw), *S.wkv_scan_backward(*pos, gy, **kw)) if t is not None]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, out))
    other, _, _ = operands(j)
    for t, n in zip(pos, other):
        t.copy_(n)
    graph.replay()
    torch.cuda.synchronize()
    want = [t for t in (*S.wkv_scan_forward(*pos, **kw), *S.wkv_scan_backward(*pos, gy, **kw)) if t is not None]
    assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("T", [1, 17, 300])
def test_rate_of_minus_infinity(S, T):
    """A state with A = -inf forgets at every token, as with any rate whose
    decay is 0, whether or not the last tile is whole."""
    C, N = 64, 16
    i = draw("f32", (2, T), C, N, 1, seed=T)
    pos, kw, _ = operands(i)
    runs = []
    for rate in (float("-inf"), -1e30):
        pos[2] = dev(i["A"])
        pos[2][::3, 1::4] = rate
        y, fin, ck = S.wkv_scan_forward(*pos, init_state=dev(i["h0"]), want_ckpt=True, **kw)
        grads = S.wkv_scan_backward(*pos, dev(i["gy"]), init_state=dev(i["h0"]), g_final=dev(i["gf"]), ckpt=ck,
                                    want_g_init=True, **kw)
        state = dev(i["h0"])
        one = S.wkv_scan_decode_step(*(a[:, 0].contiguous() for a in pos[:2]), pos[2],
                                     *(a[:, 0].contiguous() for a in pos[3:]), state, **{**kw, "z": kw["z"][:, 0].contiguous()})
        runs.append([y, fin, *grads, one, state])
    for a, b in zip(*runs):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("dtype,B,T,C,N,G", [("bf16", 20, 121, 1024, 16, 1), ("f32", 20, 160, 1024, 12, 1),
                                             ("f32", 5, 150, 1024, 64, 1), ("bf16", 10, 200, 1024, 32, 2),
                                             ("bf16", 10, 130, 4096, 8, 1)])
def test_backward_of_more_than_one_wave(S, O, dtype, B, T, C, N, G):
    """CTAs for a little more than one wave: the last sequences are cut along T
    and the others are not. The last three against the oracle; the parameter
    gradients against its sums and those of a call on the others."""
    i = draw(dtype, (B, T), C, N, G, seed=N)
    pos, kw, ref = operands(i)
    h0, gf, k = dev(i["h0"]), dev(i["gf"]), B - 3
    _, _, ckpt = S.wkv_scan_forward(*pos, **kw, init_state=h0, want_ckpt=True)
    got = dict(zip(NAMES, S.wkv_scan_backward(*pos, dev(i["gy"]), **kw, init_state=h0, g_final=gf, ckpt=ckpt, want_g_init=True)))
    again = S.wkv_scan_backward(*pos, dev(i["gy"]), **kw, init_state=h0, g_final=gf, want_g_init=True)
    assert all(torch.equal(a, b) for a, b in zip(got.values(), again))
    head = [a if a.dim() == 2 else a[:k] for a in pos]
    rest = dict(zip(NAMES, S.wkv_scan_backward(*head, dev(i["gy"])[:k], **{**kw, "z": kw["z"][:k]}, init_state=h0[:k],
                                               g_final=gf[:k], want_g_init=True)))
    ref = {n: a[k:] if n in ("x", "dt", "Bm", "Cm", "z") else a for n, a in ref.items()}
    want = O.scan_backward(gy=i["gy32"][k:], init_state=i["h0"][k:], g_final=i["gf"][k:], **ref)
    for n in NAMES:
        if n in ("gA", "gD", "gdt_bias"):
            assert rel_err(host64(got[n]), want[n] + host64(rest[n])) < 2 * TOL32, n  # of both sides
        else:
            tol = TOL32 if got[n].dtype == torch.float32 else TOL["bf16"]
            assert rel_err(host64(got[n][k:]), want[n]) < tol, n
            assert rel_err(host64(got[n][:k]), host64(rest[n])) < 2 * tol, n
