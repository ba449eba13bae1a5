"""Measured cases of the state-space operators: the short causal convolution, the per-head norm with position rotation,
and the selective scan, each in training (forward and backward), over prompts and for single tokens.

With ``own`` false, ``run`` computes the operators from elementary torch operations; with ``own`` true it calls the
library (``rwkv_wkv_linear_mix_b200.ssm``) the way a user does.
"""

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one training step of the block's convolution, a long batch
        dict(name="conv train bf16", op="conv", mode="train", dtype="bf16", B=8, T=4096, C=4096, W=4, silu=True, bias=True),
        # the prompts of 32 slots, some of them empty, in one call
        dict(name="conv slots f32", op="conv", mode="slots", dtype="f32", S=32, longest=512, C=2560, W=4, silu=True, bias=True),
        # a new token for every slot of a small model: nothing but latency
        dict(name="conv decode f32", op="conv", mode="decode", dtype="f32", S=32, C=768, W=4, silu=True, bias=True),
        # queries and keys of a training batch, all heads rotated
        dict(name="norm train bf16", op="norm", mode="train", dtype="bf16", B=8, T=4096, Hq=32, Hk=32, K=64, R=64, interleaved=False),
        # an odd prompt: shared key heads, only a part of each head rotated
        dict(name="norm train f32 odd", op="norm", mode="train", dtype="f32", B=3, T=777, Hq=5, Hk=2, K=80, R=48, interleaved=True),
        # a new token for every slot, far positions
        dict(name="norm decode bf16", op="norm", mode="decode", dtype="bf16", S=32, Hq=32, Hk=8, K=128, R=128, interleaved=False),
        # one training step of the scan
        dict(name="scan train bf16", op="scan", mode="train", dtype="bf16", B=8, T=2048, C=2560, N=16, G=1, z=True),
        # an odd training batch in full precision: wide state, two groups, no gate
        dict(name="scan train f32 odd", op="scan", mode="train", dtype="f32", B=2, T=513, C=776, N=64, G=2, z=False),
        # a single long prompt of a small model: few channels, so the length has to carry the parallelism
        dict(name="scan prompt f32", op="scan", mode="prompt", dtype="f32", B=1, T=8191, C=1536, N=16, G=1, z=True),
        # a batch of prompts
        dict(name="scan prompt bf16", op="scan", mode="prompt", dtype="bf16", B=8, T=2048, C=4096, N=16, G=1, z=True),
        # the prompts of 32 slots in one call
        dict(name="scan slots bf16", op="scan", mode="slots", dtype="bf16", S=32, longest=512, C=4096, N=16, G=1, z=True),
        # a new token for every one of 256 slots: the state goes through once
        dict(name="scan decode bf16", op="scan", mode="decode", dtype="bf16", S=256, C=4096, N=16, G=1, z=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "norm", "scan", "scan"])
    dtype = rng.choice(["f32", "bf16"])
    unit = 8 if dtype == "bf16" else 4
    c = dict(op=op, dtype=dtype)
    if op == "norm":
        c["mode"] = rng.choice(["train", "train", "decode"])
        K = rng.choice([16, 32, 64, 80, 96, 128, 192, 256])
        c.update(K=K, Hq=_spread(rng, 1, 40), Hk=_spread(rng, 1, 16), interleaved=rng.random() < 0.4)
        c["R"] = 16 * rng.randint(1, K // 16)
        if c["mode"] == "decode":
            c["S"] = _spread(rng, 1, 512)
        else:
            c["B"] = _spread(rng, 1, 16)
            row = c["B"] * (c["Hq"] + c["Hk"]) * K
            c["T"] = _spread(rng, 1, max(1, min(8192, (1 << 26) // row)))
        return c
    c["mode"] = rng.choice(["train", "slots", "decode"] if op == "conv" else ["train", "train", "prompt", "slots", "decode"])
    C = unit * _spread(rng, 2, 5120 // unit)
    if op == "conv":
        c.update(W=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7, bias=rng.random() < 0.7)
        most = 1 << 26
    else:
        G = rng.choice([1, 1, 1, 2, 4])
        C = G * unit * max(1, C // (G * unit))
        N = rng.choice([8, 16, 16, 16, 24, 32, 64])
        c.update(N=N, G=G, z=rng.random() < 0.6)
        most = (1 << 28) // max(16, N)
    c["C"] = C
    if c["mode"] == "decode":
        c["S"] = _spread(rng, 1, 512)
    elif c["mode"] == "slots":
        c["S"] = _spread(rng, 1, 64)
        c["longest"] = _spread(rng, 1, max(1, min(1024, most // (c["S"] * C))))
    else:
        c["B"] = _spread(rng, 1, 8)
        c["T"] = _spread(rng, 1, max(1, min(8192, most // (c["B"] * C))))
    return c


def _lengths(case):
    """Tokens of each slot of a "slots" case: spread over 0 .. longest, about one slot in eight empty."""
    rng = random.Random(case["S"] * 100003 + case["longest"])
    lengths = [0 if rng.random() < 0.125 else rng.randint(1, case["longest"]) for _ in range(case["S"])]
    return lengths if any(lengths) else [1] + lengths[1:]


def _tokens(case):
    if case["mode"] == "slots":
        return sum(_lengths(case))
    return case["S"] if case["mode"] == "decode" else case["B"] * case["T"]


def work(case):
    """Bytes: every input read once, every output written once. Operations: those of the formulas, an exponential as one."""
    e = 2 if case["dtype"] == "bf16" else 4
    n, train = _tokens(case), case["mode"] == "train"
    if case["op"] == "norm":
        row, K = (case["Hq"] + case["Hk"]) * case["K"], case["K"]
        q = n * row * e
        if train:  # x and g in; y and gx out
            return {"bytes": 4 * q + 4 * (4 * K + case["R"] // 2), "flops": 20 * n * row}
        return {"bytes": 2 * q + 4 * (2 * K + case["R"] // 2) + 4 * n, "flops": 7 * n * row}
    C = case["C"]
    if case["op"] == "conv":
        W = case["W"]
        par = 4 * C * (W + 1)
        state = 0 if train else 2 * case["S"] * (W - 1) * C * e
        if train:  # x, g in; y, gx out
            return {"bytes": 4 * n * C * e + 2 * par, "flops": (6 * W + 12) * n * C}
        return {"bytes": 2 * n * C * e + par + state, "flops": (2 * W + 4) * n * C}
    N, G, z = case["N"], case["G"], 1 if case["z"] else 0
    par = 4 * C * (N + 2)
    bc = 2 * n * G * N * e
    if train:  # x, dt, B, C, z, gy in; y, gx, gdt, gB, gC, gz and the final state out
        return {"bytes": n * C * e * (6 + 2 * z) + 2 * bc + 2 * par + 4 * case["B"] * C * N, "flops": 22 * n * C * N}
    rows = case["B"] if case["mode"] == "prompt" else 2 * case["S"]
    return {"bytes": n * C * e * (3 + z) + bc + par + 4 * rows * C * N, "flops": 7 * n * C * N}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    s = {"case": dict(case)}
    mode = case["mode"]
    lead = (case["B"], case["T"]) if mode in ("train", "prompt") else (_tokens(case),)
    if mode == "slots":
        cu = torch.tensor([0] + _lengths(case)).cumsum(0)
        s["cu"] = cu.to(torch.int32).cuda()
    if case["op"] == "norm":
        Hq, Hk, K, R = case["Hq"], case["Hk"], case["K"], case["R"]
        if mode == "decode":
            lead = (case["S"], 1)
            s["positions"] = torch.randint(0, 1 << 20, (case["S"], 1), generator=g, device="cuda", dtype=torch.int32)
        else:
            s["positions"] = None
        s["q"], s["k"] = normal(*lead, Hq * K, std=2.0), normal(*lead, Hk * K, std=0.7)
        s["wq"], s["wk"] = uniform(K, lo=0.5, hi=1.5), uniform(K, lo=0.5, hi=1.5)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda()
        if mode == "train":
            s["gq"], s["gk"] = normal(*lead, Hq * K), normal(*lead, Hk * K)
        return s
    C = case["C"]
    s["x"] = normal(*lead, C)
    if mode == "train":
        s["gy"] = normal(*lead, C)
    if case["op"] == "conv":
        W = case["W"]
        s["w"] = uniform(W, C, lo=-W ** -0.5, hi=W ** -0.5)
        s["bias"] = uniform(C, lo=-W ** -0.5, hi=W ** -0.5) if case["bias"] else None
        if mode != "train":
            s["state"] = normal(case["S"], W - 1, C)
        return s
    N, G = case["N"], case["G"]
    # time constants of 0.001 .. 0.1 through the softplus, decay rates about 1 .. N
    step = torch.exp(uniform(C, lo=math.log(1e-3), hi=math.log(0.1)))
    s["dt_bias"] = torch.log(torch.expm1(step))
    s["dt"] = normal(*lead, C, std=0.5)
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.2 * normal(C, N, dtype=torch.float32))
    s["Bm"], s["Cm"] = normal(*lead, G * N), normal(*lead, G * N)
    s["D"] = uniform(C, lo=0.5, hi=1.5)
    s["z"] = normal(*lead, C) if case["z"] else None
    if mode in ("slots", "decode"):
        s["state"] = normal(case["S"], C, N, std=0.3, dtype=torch.float32)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return {"conv": _own_conv, "norm": _own_norm, "scan": _own_scan}[case["op"]](s, case["mode"])
    return {"conv": _plain_conv, "norm": _plain_norm, "scan": _plain_scan}[case["op"]](s, case["mode"])


def _own_conv(s, mode):
    from rwkv_wkv_linear_mix_b200 import ssm
    silu = s["case"]["silu"]
    if mode == "train":
        y = ssm.wkv_conv_forward(s["x"], s["w"], s["bias"], silu=silu)
        gx, gw, gbias, _ = ssm.wkv_conv_backward(s["x"], s["w"], s["gy"], s["bias"], silu=silu)
        out = {"y": y, "gx": gx, "gw": gw}
        return out if gbias is None else dict(out, gbias=gbias)
    if mode == "slots":
        y = ssm.wkv_conv_chunk_step(s["x"], s["w"], s["cu"], s["state"], s["bias"], silu=silu)
    else:
        y = ssm.wkv_conv_decode_step(s["x"], s["w"], s["state"], s["bias"], silu=silu)
    return {"y": y, "state": s["state"]}


def _own_norm(s, mode):
    from rwkv_wkv_linear_mix_b200 import ssm
    how = dict(head_size=s["case"]["K"], eps=EPS, interleaved=s["case"]["interleaved"])
    q, k = ssm.wkv_norm_rotate(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["positions"], **how)
    out = {"q": q, "k": k}
    if mode == "train":
        back = ssm.wkv_norm_rotate_backward(s["q"], s["k"], s["gq"], s["gk"], s["wq"], s["wk"], s["inv_freq"],
                                            s["positions"], **how)
        out.update(zip(("gq", "gk", "gwq", "gwk"), back))
    return out


def _own_scan(s, mode):
    from rwkv_wkv_linear_mix_b200 import ssm
    data = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    par = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if mode == "train":
        y, last, ckpt = ssm.wkv_scan_forward(*data, **par, want_ckpt=True)
        grads = ssm.wkv_scan_backward(*data, s["gy"], ckpt=ckpt, **par)
        names = ("gx", "gdt", "gA", "gB", "gC", "gD", "gz", "gdt_bias")
        return {"y": y, "state": last, **{n: v for n, v in zip(names, grads) if v is not None}}
    if mode == "prompt":
        y, last = ssm.wkv_scan_forward(*data, **par)
        return {"y": y, "state": last}
    if mode == "slots":
        y = ssm.wkv_scan_chunk_step(*data, s["cu"], s["state"], **par)
    else:
        y = ssm.wkv_scan_decode_step(*data, s["state"], **par)
    return {"y": y, "state": s["state"]}


# -- the plain forms ---------------------------------------------------------------------------------------------------

def _silu(x):
    return x * torch.sigmoid(x)


def _dsilu(x):
    p = torch.sigmoid(x)
    return p * (1 + x * (1 - p))


def _rows_of(cu, n):
    """Slot of each of n packed tokens, and its place within the slot."""
    t = torch.arange(n, device=cu.device)
    slot = torch.searchsorted(cu[1:].long(), t, right=True)
    return slot, t - cu.long()[slot]


def _plain_conv(s, mode):
    x, w, W = s["x"].float(), s["w"], s["case"]["W"]
    act = _silu if s["case"]["silu"] else (lambda v: v)
    bias = 0.0 if s["bias"] is None else s["bias"]
    to = s["x"].dtype
    if mode == "train":
        T = x.shape[1]
        padded = torch.nn.functional.pad(x, (0, 0, W - 1, 0))
        taps = padded.unfold(1, W, 1).transpose(-1, -2)                        # [B, T, W, C]
        pre = (taps * w).sum(-2) + bias
        g = s["gy"].float()
        gpre = g * _dsilu(pre) if s["case"]["silu"] else g
        after = torch.nn.functional.pad(gpre, (0, 0, 0, W - 1)).unfold(1, W, 1).transpose(-1, -2)
        gx = (after * w.flip(0)).sum(-2)
        gw = (taps * gpre.unsqueeze(-2)).sum((0, 1), dtype=torch.float64).float() if T else torch.zeros_like(w)
        out = {"y": act(pre).to(to), "gx": gx.to(to), "gw": gw}
        return out if s["bias"] is None else dict(out, gbias=gpre.sum((0, 1), dtype=torch.float64).float())
    state = s["state"]
    S, n = state.shape[0], x.shape[0]
    cu = s["cu"].long() if mode == "slots" else torch.arange(S + 1, device=x.device)
    # every slot's window: its state, then its tokens, all packed in one array
    every = torch.cat((state.float().reshape(-1, x.shape[-1]), x))
    slot, place = _rows_of(cu, n)
    back = place[:, None] + torch.arange(1 - W, 1, device=x.device)            # place of each tap, below 0 in the state
    first = cu[slot][:, None]
    at = torch.where(back < 0, slot[:, None] * (W - 1) + back + W - 1, S * (W - 1) + first + back)
    y = act((every[at] * w).sum(1) + bias).to(to)
    end = cu[1:, None] - cu[:-1, None] + torch.arange(1 - W, 0, device=x.device)
    each = torch.arange(S, device=x.device)[:, None]
    at = torch.where(end < 0, each * (W - 1) + end + W - 1, S * (W - 1) + cu[:-1, None] + end)
    state.copy_(every[at])
    return {"y": y, "state": state}


def _angles(s, mode):
    T = s["q"].shape[1]
    p = torch.arange(T, device="cuda")[None] if s["positions"] is None else s["positions"]
    a = p[..., None].double() * s["inv_freq"].double()                         # far positions need 64 bits
    return torch.cos(a).float()[:, :, None], torch.sin(a).float()[:, :, None]  # [., T, 1, R/2]


def _rotate(v, cos, sin, R, interleaved):
    r, rest = v[..., :R], v[..., R:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else r.chunk(2, -1)
    c, d = a * cos - b * sin, a * sin + b * cos
    r = torch.stack((c, d), -1).flatten(-2) if interleaved else torch.cat((c, d), -1)
    return torch.cat((r, rest), -1)


def _plain_norm(s, mode):
    K, R, il = s["case"]["K"], s["case"]["R"], s["case"]["interleaved"]
    cos, sin = _angles(s, mode)

    def forward(x, w):
        v = x.float().unflatten(-1, (-1, K))
        r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        return _rotate(v * r * w, cos, sin, R, il).flatten(-2).to(x.dtype)

    def backward(x, w, g):
        v = x.float().unflatten(-1, (-1, K))
        r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        gn = _rotate(g.float().unflatten(-1, (-1, K)), cos, -sin, R, il)
        gw = (gn * (v * r)).sum((0, 1, 2), dtype=torch.float64).float()
        gv = gn * w
        return (r * (gv - v * r.square() * (gv * v).mean(-1, keepdim=True))).flatten(-2).to(x.dtype), gw

    out = {"q": forward(s["q"], s["wq"]), "k": forward(s["k"], s["wk"])}
    if mode == "train":
        out["gq"], out["gwq"] = backward(s["q"], s["wq"], s["gq"])
        out["gk"], out["gwk"] = backward(s["k"], s["wk"], s["gk"])
    return out


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h_{-1} = 0, in doubling steps."""
    shift = 1
    while shift < a.shape[1]:
        b = torch.cat((b[:, :shift], torch.addcmul(b[:, shift:], a[:, shift:], b[:, :-shift])), 1)
        a = torch.cat((a[:, :shift], a[:, shift:] * a[:, :-shift]), 1)
        shift *= 2
    return b


def _softplus(x):
    return torch.relu(x) + torch.log1p(torch.exp(-x.abs()))


def _plain_scan(s, mode):
    G, C, N = s["case"]["G"], s["case"]["C"], s["case"]["N"]
    to = s["x"].dtype
    batched = mode in ("train", "prompt")
    lift = (lambda v: v.float()) if batched else (lambda v: v.float()[None])   # [B, T, .]
    x, raw = lift(s["x"]), lift(s["dt"]) + s["dt_bias"]
    dt = _softplus(raw)
    Bm = lift(s["Bm"]).unflatten(-1, (G, 1, N))
    Cm = lift(s["Cm"]).unflatten(-1, (G, 1, N))
    A, grouped = s["A"], (lambda v: v.unflatten(2, (G, C // G)))               # [B, T, C, .] -> [B, T, G, C/G, .]
    a = torch.exp(dt[..., None] * A)
    b = (grouped((dt * x)[..., None]) * Bm).flatten(2, 3)
    if not batched:
        # packed slots: a slot's first token starts over from its state
        n, state = x.shape[1], s["state"]
        cu = s["cu"].long() if mode == "slots" else torch.arange(state.shape[0] + 1, device=x.device)
        slot, place = _rows_of(cu, n)
        first = (place == 0)[None, :, None, None]
        b = torch.where(first, torch.addcmul(b, a, state[slot][None]), b)
        a = torch.where(first, 0.0, a)
    h = _scan(a, b)
    y = (grouped(h) * Cm).sum(-1).flatten(2, 3) + s["D"] * x
    gate = _silu(lift(s["z"])) if s["z"] is not None else None
    out = (y * gate if gate is not None else y).to(to)
    if not batched:
        if n:
            some = (cu[1:] > cu[:-1])[:, None, None]
            state.copy_(torch.where(some, h[0][(cu[1:] - 1).clamp(min=0)], state))
        return {"y": out[0], "state": state}
    out = {"y": out, "state": h[:, -1].clone()}
    if mode == "prompt":
        return out
    gy = s["gy"].float()
    gs = gy * gate if gate is not None else gy
    ah = a * torch.cat((torch.zeros_like(h[:, :1]), h[:, :-1]), 1)             # a_t h_{t-1}
    gC = (grouped(h) * grouped(gs[..., None])).sum(3).flatten(-2)
    del h
    q = (grouped(gs[..., None]) * Cm).flatten(2, 3)
    # G_t = q_t + a_{t+1} G_{t+1}
    nxt = torch.cat((a[:, 1:], torch.zeros_like(a[:, :1])), 1)
    Gh = _scan(nxt.flip(1), q.flip(1)).flip(1)
    del nxt, q
    gB = (grouped(Gh) * grouped((dt * x)[..., None])).sum(3).flatten(-2)
    GB = (grouped(Gh) * Bm).sum(-1).flatten(2, 3)
    ah.mul_(Gh)
    graw = (GB * x + (ah * A).sum(-1)) * torch.sigmoid(raw)
    out.update(gx=(GB * dt + gs * s["D"]).to(to), gdt=graw.to(to), gA=(ah * dt[..., None]).sum((0, 1), dtype=torch.float64).float(),
               gB=gB.to(to), gC=gC.to(to), gD=(gs * x).sum((0, 1), dtype=torch.float64).float())
    if gate is not None:
        out["gz"] = (gy * y * _dsilu(lift(s["z"]))).to(to)
    out["gdt_bias"] = graw.sum((0, 1), dtype=torch.float64).float()
    return out


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, token by token
# ---------------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    d = {n: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for n, v in s.items()}
    return {"conv": _exact_conv, "norm": _exact_norm, "scan": _exact_scan}[case["op"]](d, case)


def _exact_conv(d, case):
    W, x, w = case["W"], d["x"], d["w"]
    sg = torch.sigmoid
    if case["mode"] == "train":
        x = x.requires_grad_()
        w = w.requires_grad_()
        bias = d["bias"].requires_grad_() if case["bias"] else torch.zeros(case["C"], device="cuda", dtype=torch.float64)
        pre = bias.expand_as(x)
        for j in range(W):  # tap j sees the token W-1-j back
            lag = W - 1 - j
            if lag < case["T"]:
                past = x[:, :case["T"] - lag] * w[j]
                pre = pre + torch.cat((torch.zeros_like(x[:, :lag]), past), 1)
        y = pre * sg(pre) if case["silu"] else pre
        grads = torch.autograd.grad(y, [x, w] + ([bias] if case["bias"] else []), d["gy"])
        return dict(zip(("y", "gx", "gw", "gbias"), (y.detach(),) + grads))
    ys, states = [], []
    lengths = _lengths(case) if case["mode"] == "slots" else [1] * case["S"]
    at = 0
    for i, n in enumerate(lengths):
        win = torch.cat((d["state"][i], x[at:at + n]))
        at += n
        pre = sum(win[j:j + n] * w[j] for j in range(W)) + (d["bias"] if case["bias"] else 0.0)
        ys.append(pre * sg(pre) if case["silu"] else pre)
        states.append(win[n:])
    return {"y": torch.cat(ys), "state": torch.stack(states)}


def _exact_norm(d, case):
    K, R, T = case["K"], case["R"], d["q"].shape[1]
    p = torch.arange(T, device="cuda")[None] if d["positions"] is None else d["positions"]
    turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), p.double()[:, :, None, None] * d["inv_freq"])

    def of(x, w):
        v = x.reshape(*x.shape[:2], -1, K)
        v = v / torch.sqrt((v * v).sum(-1, keepdim=True) / K + EPS) * w
        r = v[..., :R]
        if case["interleaved"]:
            c = torch.view_as_complex(r.reshape(*r.shape[:-1], R // 2, 2).contiguous()) * turn
            r = torch.view_as_real(c).reshape(r.shape)
        else:
            c = torch.complex(r[..., :R // 2], r[..., R // 2:]) * turn
            r = torch.cat((c.real, c.imag), -1)
        return torch.cat((r, v[..., R:]), -1).reshape(x.shape)

    out = {}
    for n in ("q", "k"):
        x, w = d[n].requires_grad_(), d["w" + n].requires_grad_()
        y = of(x, w)
        out[n] = y.detach()
        if case["mode"] == "train":
            out["g" + n], out["gw" + n] = torch.autograd.grad(y, [x, w], d["g" + n])
    return out


def _exact_scan(d, case):
    G, C, N, mode = case["G"], case["C"], case["N"], case["mode"]
    A, D = d["A"], d["D"]
    wide = lambda v: v.reshape(-1, G, 1, N).expand(-1, G, C // G, N).reshape(-1, C, N)  # noqa: E731
    raw = d["dt"] + d["dt_bias"]
    dt = torch.nn.functional.softplus(raw, threshold=700)
    gate = d["z"] * torch.sigmoid(d["z"]) if case["z"] else torch.ones_like(d["x"])
    if mode in ("slots", "decode"):
        h = d["state"].clone()
        y = torch.empty_like(d["x"])
        lengths = torch.tensor(_lengths(case) if mode == "slots" else [1] * case["S"], device="cuda")
        start = lengths.cumsum(0) - lengths
        for t in range(int(lengths.max()) if len(lengths) else 0):
            on = (lengths > t).nonzero()[:, 0]
            i = start[on] + t
            h[on] = torch.exp(dt[i][..., None] * A) * h[on] + (dt[i] * d["x"][i])[..., None] * wide(d["Bm"][i])
            y[i] = ((h[on] * wide(d["Cm"][i])).sum(-1) + D * d["x"][i]) * gate[i]
        return {"y": y, "state": h}
    B, T, x = case["B"], case["T"], d["x"]
    if mode == "train" and B * T * C * N > 1 << 30:
        return None
    keep = torch.empty((T, B, C, N) if mode == "train" else (0,), device="cuda", dtype=torch.float64)
    h = torch.zeros((B, C, N), device="cuda", dtype=torch.float64)
    s = torch.empty_like(x)
    for t in range(T):
        h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * x[:, t])[..., None] * wide(d["Bm"][:, t])
        s[:, t] = (h * wide(d["Cm"][:, t])).sum(-1) + D * x[:, t]
        if mode == "train":
            keep[t] = h
    out = {"y": s * gate, "state": h}
    if mode == "prompt":
        return out
    gs = d["gy"] * gate
    gx, gdt = torch.empty_like(x), torch.empty_like(x)
    gB, gC = torch.empty_like(d["Bm"]), torch.empty_like(d["Cm"])
    gA, back = torch.zeros_like(A), torch.zeros_like(h)
    per_group = lambda v: v.reshape(B, G, C // G, N).sum(2).reshape(B, G * N)  # noqa: E731
    for t in range(T - 1, -1, -1):
        a = torch.exp(dt[:, t, :, None] * A)
        prev = keep[t - 1] if t else torch.zeros_like(h)
        gC[:, t] = per_group(gs[:, t, :, None] * keep[t])
        back = back + gs[:, t, :, None] * wide(d["Cm"][:, t])
        gB[:, t] = per_group(back * (dt[:, t] * x[:, t])[..., None])
        gb = (back * wide(d["Bm"][:, t])).sum(-1)
        gx[:, t] = gb * dt[:, t] + gs[:, t] * D
        gdt[:, t] = gb * x[:, t] + (back * prev * a * A).sum(-1)
        gA += (back * prev * a * dt[:, t, :, None]).sum(0)
        back = back * a
    graw = gdt * torch.sigmoid(raw)
    out.update(gx=gx, gdt=graw, gA=gA, gB=gB, gC=gC, gD=(gs * x).sum((0, 1)))
    if case["z"]:
        p = torch.sigmoid(d["z"])
        out["gz"] = d["gy"] * s * p * (1 + d["z"] * (1 - p))
    out["gdt_bias"] = graw.sum((0, 1))
    return out
