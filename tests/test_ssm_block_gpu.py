"""The state-space operators together, as a block uses them: the convolution
makes x, a norm with rotation prepares C and B, the scan mixes; training
(forward and every gradient) against the fp64 oracle, and a prompt followed by
single tokens against the whole sequence. And the norm with rotation ahead of
the head-state recurrence.

Tolerances: the operators' own (tests of each) added up along the chain, in
float32 throughout: 1e-5 + 2e-5 + 1.2e-4 with amplification by the scan's
derivative in its inputs of order one; held to 5e-4."""

import numpy as np
import pytest
import torch

from _dev import dev, host64, need_gpu, rel_err

pytestmark = pytest.mark.gpu
TOL = 5e-4


@pytest.fixture(scope="module")
def S():
    need_gpu()
    from rwkv_wkv_linear_mix_b200 import ssm
    return ssm


@pytest.fixture(scope="module")
def O():
    from oracle import ssm
    return ssm


B, T, C, N, G, W = 2, 150, 64, 16, 2, 4
FREQ = (100.0 ** (-np.arange(0, N, 2) / N)).astype(np.float32)


def draw():
    rng = np.random.Generator(np.random.PCG64(0))
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    i = dict(u=f(B, T, C), dt=0.5 * f(B, T, C), z=f(B, T, C), Bm=f(B, T, G * N), Cm=f(B, T, G * N), gy=f(B, T, C),
             w=rng.uniform(-1, 1, size=(W, C)).astype(np.float32), bias=0.1 * f(C), wb=1 + 0.1 * f(N), wc=1 + 0.1 * f(N),
             D=1 + 0.1 * f(C), A=(-np.arange(1, N + 1) * np.exp(0.2 * f(C, N))).astype(np.float32))
    i["dt_bias"] = np.log(np.expm1(np.exp(rng.uniform(np.log(1e-2), np.log(0.3), size=C)))).astype(np.float32)
    return i


def test_training_step(S, O):
    i = draw()
    t = {n: dev(a) for n, a in i.items()}
    f = dev(FREQ)
    x = S.wkv_conv_forward(t["u"], t["w"], t["bias"])
    Cr, Br = S.wkv_norm_rotate(t["Cm"], t["Bm"], t["wc"], t["wb"], f, head_size=N)
    scan = (x, t["dt"], t["A"], Br, Cr)
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"])
    y, _, ckpt = S.wkv_scan_forward(*scan, **kw, want_ckpt=True)
    gx, gdt, gA, gBr, gCr, gD, gz, gdb, _ = S.wkv_scan_backward(*scan, t["gy"], **kw, ckpt=ckpt)
    gC, gB, gwc, gwb = S.wkv_norm_rotate_backward(t["Cm"], t["Bm"], gCr, gBr, t["wc"], t["wb"], f, head_size=N)
    gu, gw, gbias, _ = S.wkv_conv_backward(t["u"], t["w"], gx, t["bias"])

    pos = np.broadcast_to(np.arange(T), (B, T))
    rx = O.conv_forward(i["u"], i["w"], i["bias"])
    rB, rC = (O.norm_rotate(i[n], i[w], FREQ, pos, N, 1e-6, False) for n, w in (("Bm", "wb"), ("Cm", "wc")))
    ref = dict(x=rx, dt=i["dt"], A=i["A"], Bm=rB, Cm=rC, D=i["D"], z=i["z"], dt_bias=i["dt_bias"])
    assert rel_err(host64(y), O.scan_forward(**ref)[0]) < TOL
    g = O.scan_backward(gy=i["gy"], **ref)
    want = dict(zip(("gu", "gw", "gbias"), O.conv_backward(i["u"], i["w"], g["gx"], i["bias"])))
    want["gB"], want["gwb"] = O.norm_rotate_backward(i["Bm"], g["gB"], i["wb"], FREQ, pos, N, 1e-6, False)
    want["gC"], want["gwc"] = O.norm_rotate_backward(i["Cm"], g["gC"], i["wc"], FREQ, pos, N, 1e-6, False)
    want.update({n: g[n] for n in ("gdt", "gA", "gD", "gz", "gdt_bias")})
    got = dict(gu=gu, gw=gw, gbias=gbias, gB=gB, gwb=gwb, gC=gC, gwc=gwc, gdt=gdt, gA=gA, gD=gD, gz=gz, gdt_bias=gdb)
    for n, a in got.items():
        assert rel_err(host64(a), want[n]) < TOL, n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_then_single_tokens(S, dtype):
    """100 tokens as slots, then 50 single tokens, through all three operators:
    the bits of one call over the 150 (slots are never cut along T)."""
    i = draw()
    t = {n: dev(a) for n, a in i.items()}
    for n in ("u", "dt", "z", "Bm", "Cm"):
        t[n] = t[n].to(dtype)
    f, kw = dev(FREQ), dict(D=t["D"], dt_bias=t["dt_bias"])

    def slots(a, b, conv, state):
        n = b - a
        flat = {k: t[k][:, a:b].reshape(B * n, -1).contiguous() for k in ("u", "dt", "z", "Bm", "Cm")}
        cu = (n * torch.arange(B + 1, dtype=torch.int32)).cuda()
        pos = torch.arange(a, b, dtype=torch.int32).repeat(B, 1).cuda()
        x = S.wkv_conv_chunk_step(flat["u"], t["w"], cu, conv, t["bias"])
        Cr, Br = S.wkv_norm_rotate(flat["Cm"].view(B, n, -1), flat["Bm"].view(B, n, -1), t["wc"], t["wb"], f, pos, head_size=N)
        return S.wkv_scan_chunk_step(x, flat["dt"], t["A"], Br.view(B * n, -1), Cr.view(B * n, -1), cu, state, z=flat["z"],
                                     **kw).view(B, n, C)

    def fresh():
        return torch.zeros(B, W - 1, C, device="cuda", dtype=dtype), torch.zeros(B, C, N, device="cuda")

    conv, state = fresh()
    whole = slots(0, T, conv, state)
    conv2, state2 = fresh()
    parts = [slots(0, 100, conv2, state2)]
    for p in range(100, T):
        tok = {k: t[k][:, p].contiguous() for k in ("u", "dt", "z", "Bm", "Cm")}
        x = S.wkv_conv_decode_step(tok["u"], t["w"], conv2, t["bias"])
        Cr, Br = S.wkv_norm_rotate(tok["Cm"][:, None], tok["Bm"][:, None], t["wc"], t["wb"], f, pos_offset=p, head_size=N)
        parts.append(S.wkv_scan_decode_step(x, tok["dt"], t["A"], Br[:, 0], Cr[:, 0], state2, z=tok["z"], **kw)[:, None])
    assert torch.equal(torch.cat(parts, 1), whole)
    assert torch.equal(conv, conv2) and torch.equal(state, state2)


def test_norm_rotate_ahead_of_the_head_state_recurrence(S, O, oracle):
    """r and k of wkv6_forward through the norm with rotation, against the two
    oracles in turn on the rounded r and k (2e-2: the recurrence's bf16 bound)."""
    from rwkv_wkv_linear_mix_b200 import wkv
    rng = np.random.default_rng(1)
    b, n, H, K = 1, 70, 2, 64
    f32 = lambda: rng.standard_normal((b, n, H * K)).astype(np.float32)  # noqa: E731
    r, k, v = (torch.from_numpy(f32()).cuda().bfloat16() for _ in range(3))
    w = torch.exp(-torch.exp(torch.from_numpy(f32()).cuda() * 0.5 - 1)).bfloat16()
    u = torch.from_numpy(rng.uniform(-1, 1, size=H * K).astype(np.float32)).cuda()
    freq = (10000.0 ** (-np.arange(0, K, 2) / K)).astype(np.float32)
    rr, kk = S.wkv_norm_rotate(r, k, inv_freq=dev(freq), head_size=K)
    pos = np.arange(n)[None]
    assert rel_err(host64(rr), O.norm_rotate(host64(r), None, freq, pos, K, 1e-6, False)) < 2.0 ** -8 + 1e-5
    o, _ = wkv.wkv6_forward(rr, kk, v, w, u)
    want, _ = oracle.wkv6_forward(host64(rr), host64(kk), host64(v), host64(w), host64(u).reshape(H, K))
    assert rel_err(host64(o), want) < 2e-2


def test_slots_and_single_tokens_in_a_graph(S):
    """A captured step over slots and one of single tokens, replayed: each
    replay moves the states on as an eager call does."""
    i = draw()
    t = {n: dev(a) for n, a in i.items()}
    n = 7
    tok = {k: t[k][:, :n].reshape(B * n, -1).contiguous() for k in ("u", "dt", "z", "Bm", "Cm")}
    one = {k: t[k][:, n].contiguous() for k in ("u", "dt", "z", "Bm", "Cm")}
    cu, kw = (n * torch.arange(B + 1, dtype=torch.int32)).cuda(), dict(D=t["D"], dt_bias=t["dt_bias"])

    def step(conv, state):
        x = S.wkv_conv_chunk_step(tok["u"], t["w"], cu, conv, t["bias"])
        a = S.wkv_scan_chunk_step(x, tok["dt"], t["A"], tok["Bm"], tok["Cm"], cu, state, z=tok["z"], **kw)
        x = S.wkv_conv_decode_step(one["u"], t["w"], conv, t["bias"])
        return a, S.wkv_scan_decode_step(x, one["dt"], t["A"], one["Bm"], one["Cm"], state, z=one["z"], **kw)

    conv, state = torch.zeros(B, W - 1, C, device="cuda"), torch.zeros(B, C, N, device="cuda")
    want = [step(conv, state) for _ in range(3)]
    conv2, state2 = torch.zeros_like(conv), torch.zeros_like(state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(conv2, state2)
    assert not conv2.any() and not state2.any()
    for a, b in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], a) and torch.equal(got[1], b)
    assert torch.equal(conv, conv2) and torch.equal(state, state2) and S.device_error() == 0


def test_two_streams_at_once(S):
    """The same calls on two streams together give what they give alone."""
    i = draw()
    t = {n: dev(a) for n, a in i.items()}
    data, kw = (t["u"], t["dt"], t["A"], t["Bm"], t["Cm"]), dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"])
    alone = [S.wkv_scan_backward(*data, t["gy"], **kw), S.wkv_conv_backward(t["u"], t["w"], t["gy"], t["bias"])]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append([S.wkv_scan_backward(*data, t["gy"], **kw), S.wkv_conv_backward(t["u"], t["w"], t["gy"], t["bias"])])
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(alone, o):
            assert all(p is None and q is None or torch.equal(p, q) for p, q in zip(a, b))
