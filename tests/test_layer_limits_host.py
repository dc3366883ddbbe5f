"""Host side of the operators around the recurrence: limits of their sizes,
refused before anything is launched (fake pointers, no GPU)."""
import pytest

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
