"""Limits of the state-space operators that are refused on the host, before
the CUDA runtime is touched."""

import pytest

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    from rwkv_wkv_linear_mix_b200 import build
    build.build()
    from rwkv_wkv_linear_mix_b200 import ssm, wkv  # noqa: F401  (ssm sets the signatures)
    return wkv.lib()


def test_positions_beyond_what_float64_holds(L):
    far = 1 << 53

    def forward(offset, T=3, R=16, q=None, positions=None):
        return L.wkv_norm_rotate(1, T, 1, 0, 16, R, 0, q, None, None, None, 1e-6, FAKE, positions, offset, 0, FAKE, None, None)

    def backward(offset, T=3):
        return L.wkv_norm_rotate_backward(1, T, 1, 0, 16, 16, 0, None, None, FAKE, None, None, None, 1e-6, FAKE, None, offset, 0,
                                          FAKE, None, None, None, FAKE, 1 << 20, None)

    for f in (forward, backward):
        for offset in (far - 2, far, (1 << 63) - 1, -far - 1, -(1 << 63)):
            assert f(offset) == 2 and b"2^53" in L.wkv_last_error()
        for offset in (far - 3, -far, 0):  # these get as far as the missing q
            assert f(offset) == 1 and b"q is NULL" in L.wkv_last_error()
    assert forward(far, R=0) == 1 and b"q is NULL" in L.wkv_last_error()             # nothing turns
    assert forward(far, positions=FAKE) == 1 and b"q is NULL" in L.wkv_last_error()  # not read


def test_launches_cut_along_T(L):
    """Few CTAs (32 channels each at N = 16) are cut, those that fill the SMs
    are not: fewer than three for two SMs in the forward."""
    ws = L.wkv_scan_forward_workspace_bytes
    assert ws(1, 4096, 32 * 221, 16, 1) > 0 and ws(1, 4096, 32 * 222, 16, 1) == 0
    assert ws(2, 2048, 4096, 16, 1) == 0 and ws(2, 2048, 2560, 16, 1) > 0
    assert ws(1, 64, 64, 16, 1) == 0  # too short to cut


@pytest.mark.parametrize("offset", [1 << 63, (1 << 64) + 5, -(1 << 63) - 1])
def test_an_offset_past_64_bits_is_not_wrapped(L, offset):
    from rwkv_wkv_linear_mix_b200 import ssm
    for f in (lambda: ssm.wkv_norm_rotate(None, None, head_size=8, pos_offset=offset),
              lambda: ssm.wkv_norm_rotate_backward(None, None, None, None, head_size=8, pos_offset=offset)):
        with pytest.raises(ValueError, match="64 bits"):
            f()
