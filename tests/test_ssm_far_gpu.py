"""State-space operators over tensors of more than 2^31 elements: what they
write at the far end has the bits of a call over the last tokens alone."""

import pytest
import torch

from _dev import need_gpu

pytestmark = pytest.mark.gpu

C, HEAD, TAIL = 16384, 1 << 17, 100  # channels enough that no launch is cut along T; the tail starts a tile


@pytest.fixture(scope="module")
def S():
    need_gpu()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    from rwkv_wkv_linear_mix_b200 import ssm
    yield ssm
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def x(S):
    torch.manual_seed(0)
    x = torch.empty(1, HEAD + TAIL, C, device="cuda", dtype=torch.bfloat16).normal_()
    assert x.numel() > 1 << 31
    return x


def tail(t, keep=0):
    return t[:, HEAD - keep:].contiguous()


def test_convolution(S, x):
    w = torch.rand(4, C, device="cuda")
    xt, prev = tail(x), tail(x, 3)[:, :3].contiguous()
    want = S.wkv_conv_forward(xt, w, None, prev)
    assert torch.equal(tail(S.wkv_conv_forward(x, w)), want)
    state = torch.cat([torch.zeros_like(prev), prev])
    cu = torch.tensor([0, HEAD, HEAD + TAIL], dtype=torch.int32).cuda()
    assert torch.equal(S.wkv_conv_chunk_step(x[0], w, cu, state)[HEAD:], want[0])
    assert torch.equal(state[1], x[0, -3:]) and torch.equal(state[0], x[0, HEAD - 3:HEAD])
    del want
    far = S.wkv_conv_backward(x, w, x)[0]
    assert torch.equal(tail(far), S.wkv_conv_backward(xt, w, xt, None, prev)[0])


def test_norm(S, x):
    f = 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    xt, how = tail(x), dict(inv_freq=f, head_size=64)
    far, _ = S.wkv_norm_rotate(x, None, **how)
    assert torch.equal(tail(far), S.wkv_norm_rotate(xt, None, pos_offset=HEAD, **how)[0])
    del far
    far = S.wkv_norm_rotate_backward(x, None, x, None, **how)[0]
    assert torch.equal(tail(far), S.wkv_norm_rotate_backward(xt, None, xt, None, pos_offset=HEAD, **how)[0])


def test_scan(S, x):
    N = 16
    A = -torch.rand(C, N, device="cuda") - 0.1
    Bm, Cm = (torch.randn(1, HEAD + TAIL, N, device="cuda").bfloat16() for _ in range(2))
    xt, bc = tail(x), (tail(Bm), tail(Cm))
    _, before = S.wkv_scan_forward(x[:, :HEAD], x[:, :HEAD], A, Bm[:, :HEAD], Cm[:, :HEAD])
    y, last, ckpt = S.wkv_scan_forward(x, x, A, Bm, Cm, want_ckpt=True)
    yt, last_t, ckpt_t = S.wkv_scan_forward(xt, xt, A, *bc, init_state=before, want_ckpt=True)
    assert torch.equal(tail(y), yt) and torch.equal(last, last_t)
    assert torch.equal(ckpt[:, HEAD // S.SCAN_CKPT_LEN:], ckpt_t)
    state = torch.cat([torch.zeros_like(before), before])
    cu = torch.tensor([0, HEAD, HEAD + TAIL], dtype=torch.int32).cuda()
    y = S.wkv_scan_chunk_step(x[0], x[0], A, Bm[0], Cm[0], cu, state)
    assert torch.equal(y[HEAD:], yt[0]) and torch.equal(state, torch.cat([before, last]))
    del y
    far = S.wkv_scan_backward(x, x, A, Bm, Cm, x, ckpt=ckpt)
    near = S.wkv_scan_backward(xt, xt, A, *bc, xt, init_state=before, ckpt=ckpt_t)
    for k in (0, 1, 3, 4):  # gx, gdt, gB, gC
        assert torch.equal(tail(far[k]), near[k]), k
