"""Host side of the operators around the recurrence: limits of their sizes,
refused before anything is launched (fake pointers, no GPU)."""
import pytest
import torch

import gated_delta_rule_158_b200 as kda

from test_layer_ops_host import CBWD, CONV, L, SBWD, SCAN, UNS, _call, at  # noqa: F401

INT_MAX = (1 << 31) - 1
MANY = [INT_MAX, INT_MAX - 1024, (1 << 31) - (1 << 16) + 1]


@pytest.mark.parametrize("num", MANY)
def test_sequence_counts_that_32_bit_loops_cannot_take(L, num):  # noqa: F811
    """A loop over num sequences in steps of 1024, and the count of sequences and
    segments, stay below 2^31: beyond that the call is refused."""
    seq = dict(cu=at(60), num=num, B=1, T=1 << 20, init=None)
    conv = dict(seq, D=8, xs=8)
    assert _call(L.kda_short_conv_fwd, CONV, dict(conv, fin=None)) == UNS
    assert _call(L.kda_short_conv_bwd, CBWD, dict(conv, dfin=None, dinit=None)) == UNS
    scan = dict(seq, D=8, xs=8, dls=8, zs=8, S=8, bs=8, cs=8, wsb=1 << 62)
    assert _call(L.kda_selective_scan_fwd, SCAN, dict(scan, fin=None)) == UNS
    assert _call(L.kda_selective_scan_bwd, SBWD, dict(scan, dfin=None, dinit=None)) == UNS
    assert kda.kda_short_conv_bwd_workspace_size(1, 1 << 20, 8, 4, num) == 0
    assert kda.kda_selective_scan_fwd_workspace_size(1, 1 << 20, 8, 8, 1, num) == 0
    assert kda.kda_selective_scan_bwd_workspace_size(1, 1 << 20, 8, 8, 1, num) == 0


def test_segments_count_towards_the_limit(L):  # noqa: F811
    num = (1 << 31) - (1 << 16)
    fits = num - (1 << 20) // 64
    assert kda.kda_selective_scan_fwd_workspace_size(1, 1 << 20, 8, 8, 1, num) == 0
    assert kda.kda_selective_scan_fwd_workspace_size(1, 1 << 20, 8, 8, 1, fits) > 8 * fits
    assert kda.kda_selective_scan_bwd_workspace_size(1, 1 << 20, 8, 8, 1, fits) > 8 * fits
    assert kda.kda_short_conv_bwd_workspace_size(1, 1 << 20, 8, 4, num) > 0


def test_binding_refuses_sizes_beyond_32_bits(monkeypatch):
    """ctypes passes the low 32 bits of an int: 2^32 + 5 tokens would be five."""
    monkeypatch.setattr(kda._lib.torch.cuda, "current_device", lambda: -1)
    many = (1 << 32) + 5
    e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    x, w, ws, A = e(1, many, 8), e(8, 4), e(256, dtype=torch.uint8), e(8, 16)
    bc, q = e(1, many, 1, 16), e(many, 1, 8)
    cu = e(many, dtype=torch.int32)
    short = e(1, 5, 8)
    for call in (lambda: kda.kda_short_conv_fwd(x, w, x, ws),
                 lambda: kda.kda_short_conv_bwd(x, w, x, dict(dx=x, dweight=w), ws),
                 lambda: kda.kda_short_conv_step(x[0], w, e(many, 3, 8), x[0]),
                 lambda: kda.kda_short_conv_fwd(short, w, short, ws, cu_seqlens=cu),
                 lambda: kda.kda_selective_scan_fwd(x, x, A, bc, bc, x, ws),
                 lambda: kda.kda_selective_scan_bwd(
                     x, x, A, bc, bc, x, dict(dx=x, ddelta=x, dA=A, dB=bc, dC=bc), ws),
                 lambda: kda.kda_selective_scan_step(x[0], x[0], A, bc[0], bc[0], e(many, 8, 16),
                                                     x[0]),
                 lambda: kda.kda_qk_norm_fwd(q, q, q, q),
                 lambda: kda.kda_qk_norm_bwd(q, q, q, q, dict(dq=q, dk=q)),
                 lambda: kda.kda_short_conv_bwd_workspace_size(1, many, 8, 4),
                 lambda: kda.kda_selective_scan_fwd_workspace_size(1, many, 8, 16),
                 lambda: kda.kda_selective_scan_bwd_workspace_size(1, 5, 8, 16, 1, many),
                 lambda: kda.kda_qk_norm_bwd_workspace_size(many, 1, 1, 8)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_binding_refuses_other_numbers_of_dimensions(monkeypatch):
    """A step of x [N, 2, D] with an output [N, D] would read the first N of its 2 N
    rows; a prompt of heads [B, T, H, D] the first B T."""
    monkeypatch.setattr(kda._lib.torch.cuda, "current_device", lambda: -1)
    e = lambda *s: torch.zeros(s)  # noqa: E731
    A, ws = e(8, 16), torch.zeros(256, dtype=torch.uint8)
    x, bc = e(3, 2, 8), e(3, 2, 1, 16)
    with pytest.raises(ValueError, match="2 dimensions"):
        kda.kda_selective_scan_step(x, x, A, bc, bc, e(3, 8, 16), e(3, 8))
    x, bc = e(1, 3, 2, 8), e(1, 3, 2, 1, 16)
    with pytest.raises(ValueError, match="3 dimensions"):
        kda.kda_selective_scan_fwd(x, x, A, bc, bc, e(1, 3, 8), ws)
    grads = dict(dx=e(1, 3, 8), ddelta=e(1, 3, 8), dA=A, dB=e(1, 3, 1, 16), dC=e(1, 3, 1, 16))
    with pytest.raises(ValueError, match="3 dimensions"):
        kda.kda_selective_scan_bwd(x, x, A, bc, bc, e(1, 3, 8), grads, ws)
