"""Host-side checks of the state-space operators' C ABI (include/wkv_ssm.h)
that need no GPU: declared, exported and bound names agree, and malformed
calls are refused before the CUDA runtime is touched."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # 16-byte aligned, never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def S():
    from rwkv_wkv_linear_mix_b200 import build
    build.build()
    from rwkv_wkv_linear_mix_b200 import ssm
    return ssm


@pytest.fixture(scope="module")
def L(S):
    from rwkv_wkv_linear_mix_b200 import wkv
    return wkv.lib()


def declared():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "wkv_ssm.h")).read(), flags=re.S)
    return {m.group(1): m.group(2).count(",") + 1
            for m in re.finditer(r"\b(wkv[A-Za-z0-9_]*)\s*\(([^;{]*?)\)\s*;", src, flags=re.S)}


def test_header_library_and_binding_agree(S):
    from rwkv_wkv_linear_mix_b200 import wkv
    lib = ctypes.CDLL(wkv.LIB_PATH)
    names = declared()
    assert set(names) == set(S.SIGNATURES)
    for n, arity in names.items():
        assert hasattr(lib, n), f"{n} declared in wkv_ssm.h but not exported"
        assert arity == len(S.SIGNATURES[n][1]), n


def test_names_are_reached_from_the_package():
    import rwkv_wkv_linear_mix_b200 as pkg
    assert pkg.wkv_scan_forward is pkg.ssm.wkv_scan_forward
    with pytest.raises(AttributeError):
        pkg.wkv_scan_nothing


def said(L, text):
    return text in L.wkv_last_error()


def test_conv_refusals(L):
    f = lambda B=2, T=4, C=8, dt=0, W=4, x=FAKE, w=FAKE, b=None, xp=None, y=FAKE: L.wkv_conv_forward(  # noqa: E731
        B, T, C, dt, W, 1, x, w, b, xp, y, None)
    assert f(B=-1) == 1 and f(dt=7) == 1
    assert f(C=6) == 2 and f(C=12, dt=1) == 2
    assert f(W=1) == 2 and f(W=5) == 2 and said(L, b"W must be")
    assert f(x=None) == 1 and said(L, b"x is NULL")
    assert f(w=FAKE + 4) == 1 and said(L, b"weight is not 16-byte aligned")
    assert f(b=FAKE + 8) == 1 and said(L, b"bias")
    assert f(xp=FAKE + 2) == 1 and said(L, b"x_prev")
    assert f(y=None) == 1 and said(L, b"y is NULL")
    assert f(B=1 << 20, T=1 << 20, C=1 << 20) == 2
    for empty in (dict(B=0), dict(T=0), dict(C=0)):
        assert f(x=None, w=None, y=None, **empty) == 0
    ws = L.wkv_conv_backward_workspace_bytes
    assert ws(2, 64, 128, 0, 4) >= 5 * 2 * 128 * 4 and ws(2, 64, 128, 0, 5) == 0 and ws(0, 64, 128, 0, 4) == 0
    b = lambda gy=FAKE, gx=FAKE, gw=FAKE, n=1 << 30: L.wkv_conv_backward(  # noqa: E731
        2, 64, 128, 0, 4, 1, FAKE, FAKE, None, None, gy, gx, gw, None, None, FAKE, n, None)
    assert b(gy=None) == 1 and said(L, b"gy is NULL")
    assert b(gw=None) == 1 and said(L, b"gweight")
    assert b(n=ws(2, 64, 128, 0, 4) - 1) == 1 and said(L, b"workspace")
    c = lambda S=2, n=4, cu=FAKE, st=FAKE, y=FAKE: L.wkv_conv_chunk_step(  # noqa: E731
        S, 8, 0, 4, 1, FAKE, FAKE, None, y, n, cu, st, None)
    assert c(n=-1) == 1 and c(S=-1) == 1
    assert c(cu=None) == 1 and said(L, b"cu_tokens")
    assert c(st=None) == 1 and said(L, b"state")
    assert c(y=None) == 1 and said(L, b"y is NULL")
    assert c(S=0, cu=None, st=None, y=None) == 0
    d = lambda x=FAKE, st=FAKE: L.wkv_conv_decode_step(2, 8, 0, 4, 1, x, FAKE, None, FAKE, st, None)  # noqa: E731
    assert d(x=None) == 1 and d(st=FAKE + 4) == 1 and said(L, b"state")


def test_norm_refusals(L):
    f = lambda B=2, T=3, Hq=2, Hk=1, K=64, R=64, dt=0, q=FAKE, k=FAKE, wq=None, eps=1e-6, fr=FAKE, po=None, il=0, \
        qo=FAKE, ko=FAKE: L.wkv_norm_rotate(B, T, Hq, Hk, K, R, dt, q, k, wq, None, eps, fr, po, 0, il, qo, ko, None)  # noqa: E731
    assert f(K=60) == 2 and f(K=264) == 2 and f(K=4) == 2 and f(K=0, R=0) == 2
    assert f(R=80) == 1 and said(L, b"R above K")
    assert f(R=24) == 2 and f(R=25, il=1) == 2 and said(L, b"R must be")
    assert f(Hq=-1) == 1 and f(dt=9) == 1
    assert f(eps=-1.0) == 1 and f(eps=float("nan")) == 1 and said(L, b"eps")
    assert f(q=None) == 1 and said(L, b"q is NULL")
    assert f(ko=None) == 1 and said(L, b"k_out")
    assert f(fr=None) == 1 and said(L, b"inv_freq")
    assert f(po=FAKE + 4) == 1 and said(L, b"positions")
    assert f(wq=FAKE + 4) == 1 and said(L, b"q_weight")
    assert f(B=1 << 20, T=1 << 20) == 2
    assert f(B=0, q=None, k=None, qo=None, ko=None, fr=None) == 0
    assert f(Hq=0, Hk=0, q=None, k=None, qo=None, ko=None, fr=None) == 0
    ws = L.wkv_norm_rotate_backward_workspace_bytes
    assert ws(2, 3, 2, 1, 64) >= 2 * 64 * 4 and ws(2, 3, 0, 0, 64) == 0 and ws(2, 3, 2, 1, 60) == 0
    b = lambda gqo=FAKE, gk=FAKE, n=1 << 30: L.wkv_norm_rotate_backward(  # noqa: E731
        2, 3, 2, 1, 64, 64, 0, FAKE, FAKE, gqo, FAKE, None, None, 1e-6, FAKE, None, 0, 0, FAKE, gk, None, None, FAKE, n, None)
    assert b(gqo=None) == 1 and said(L, b"gq_out")
    assert b(gk=None) == 1 and said(L, b"gk is NULL")
    assert b(n=16) == 1 and said(L, b"workspace")


def test_scan_refusals(L):
    def f(B=2, T=40, C=16, N=16, G=1, dt=0, x=FAKE, A=FAKE, Cm=FAKE, z=None, y=FAKE, fs=None, ck=None, ws=FAKE, n=1 << 40):
        return L.wkv_scan_forward(B, T, C, N, G, dt, x, FAKE, A, FAKE, Cm, None, z, None, 1, None, y, fs, ck, ws, n, None)

    for N in (0, 2, 6, 68, 128):
        assert f(N=N) == 2 and said(L, b"N must be")
    assert f(N=-4) == 1 and f(G=0) == 1 and f(G=3) == 1
    assert f(C=24, G=4) == 2 and f(C=24, G=2, dt=1) == 2 and said(L, b"C / G")
    assert f(C=6) == 2 and f(T=-1) == 1 and f(dt=3) == 1
    assert f(x=None) == 1 and said(L, b"x is NULL")
    assert f(A=FAKE + 4) == 1 and said(L, b"A is not")
    assert f(Cm=None) == 1 and said(L, b"Cm")
    assert f(z=FAKE + 2) == 1 and said(L, b"z is not")
    assert f(y=None) == 1 and said(L, b"all NULL")
    assert f(B=1 << 20, T=1 << 20, C=1 << 20) == 2
    assert f(B=1 << 10, T=1 << 30, C=16) == 2
    assert f(B=0, x=None) == 0 and f(C=0, x=None) == 0
    size = L.wkv_scan_forward_workspace_bytes
    assert size(16, 4096, 4096, 16, 1) == 0            # enough channels: not cut
    need = size(1, 4096, 64, 16, 1)                    # one CTA's channels: cut along T
    assert need > 0 and need % (64 * 17 * 4) == 0
    assert f(B=1, T=4096, C=64, n=need - 1) == 1 and said(L, b"workspace_bytes")
    assert f(B=1, T=4096, C=64, ws=None, n=need) == 1 and said(L, b"workspace is NULL")
    assert L.wkv_scan_ckpt_floats(2, 33, 8, 16) == 2 * 3 * 8 * 16 and L.wkv_scan_ckpt_floats(2, 0, 8, 16) == 0

    def b(gy=FAKE, gA=FAKE, z=None, gz=None, ck=FAKE, n=1 << 40, T=40):
        return L.wkv_scan_backward(2, T, 16, 16, 1, 0, FAKE, FAKE, FAKE, FAKE, FAKE, None, z, None, 1, None, gy, None, ck,
                                   FAKE, FAKE, gA, FAKE, FAKE, None, gz, None, None, FAKE, n, None)

    assert b(gy=None) == 1 and said(L, b"gy is NULL")
    assert b(gA=None) == 1 and said(L, b"gA is NULL")
    assert b(z=FAKE) == 1 and said(L, b"gz is NULL")
    size = L.wkv_scan_backward_workspace_bytes
    with_ck, without = size(2, 40, 16, 16, 1, 1), size(2, 40, 16, 16, 1, 0)
    assert without >= with_ck + 4 * L.wkv_scan_ckpt_floats(2, 40, 16, 16)
    assert b(n=with_ck - 1) == 1 and b(ck=None, n=without - 1) == 1 and said(L, b"workspace")
    c = lambda n=4, cu=FAKE, st=FAKE, y=FAKE: L.wkv_scan_chunk_step(  # noqa: E731
        2, 16, 16, 1, 0, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, 1, y, n, cu, st, None)
    assert c(n=-1) == 1 and c(cu=None) == 1 and c(st=None) == 1 and said(L, b"state")
    assert c(y=None) == 1 and said(L, b"y is NULL")
    d = lambda st=FAKE, y=FAKE: L.wkv_scan_decode_step(  # noqa: E731
        2, 16, 16, 1, 0, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, 1, y, st, None)
    assert d(st=FAKE + 4) == 1 and d(y=None) == 1


def test_binding_refuses_what_the_kernels_would_misread(S):
    """Shapes, dtypes and devices are checked before any pointer is passed."""
    import torch
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        S.wkv_conv_forward(x, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        S.wkv_norm_rotate(x, None, head_size=8)
    with pytest.raises(ValueError, match="CUDA"):
        S.wkv_scan_forward(x, x, torch.zeros(8, 16), torch.zeros(1, 4, 16), torch.zeros(1, 4, 16))
    with pytest.raises(ValueError, match="both None"):
        S.wkv_norm_rotate(None, None, head_size=8)
    with pytest.raises(ValueError, match="head_size"):
        S.wkv_norm_rotate(x, None, head_size=0)
