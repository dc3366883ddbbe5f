"""The operators around the recurrence over the ranges of their inputs on the
GPU, against the fp64 references."""
import pytest
import torch

import gated_delta_rule_158_b200 as kda

import layer_ref as R
from test_gpu_layer_edges import scan_backward, scan_forward
from test_gpu_layer_ops import (DEV, F32, flat, host, near, ok, scan_inputs, scan_opt,
                                scan_ref)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


SCAN_GRADS = dict(dx="x", ddelta="delta", dA="A", dB="Bm", dC="Cm", dD="D", dz="z",
                  ddelta_bias="delta_bias", d_init="init")


def check_scan(i, B, T, D, S, G, dtype, ref_inputs=None):
    """Forward, final state and every gradient on the reference."""
    out, fin, ws = scan_forward(i, B, T, D, S, G)
    ok(ws)
    g, ws = scan_backward(i, B, T, D, S, G)
    ok(ws)
    t, ro, rf = scan_ref(i if ref_inputs is None else ref_inputs, grad=True)
    near(flat(out), ro, dtype, "out")
    near(fin, rf, what="final")
    ((ro * host(flat(i["dout"]))).sum() + (rf * host(i["d_final"])).sum()).backward()
    for key, src in SCAN_GRADS.items():
        near(g[key].reshape(t[src].shape), t[src].grad, what=key)


@pytest.mark.parametrize("B,T,D,S,cu", [
    (2, 33, 40, 16, None),      # uncut, a tile's tokens behind the end
    (1, 700, 16, 16, None),     # cut into segments
    (1, 76, 48, 8, [0, 3, 3, 41, 76]),
])
def test_scan_states_that_keep_nothing(B, T, D, S, cu):
    """A = -inf in some states: each token forgets the one before, and nothing
    becomes NaN.  The reference takes -1e30, whose decays are 0 as well."""
    i = scan_inputs((B, T, D, S, 1, cu, True, True, True, True, True, False), F32, seed=41)
    i["A"][:, ::5] = -float("inf")
    i["A"][3] = -torch.finfo(F32).max  # its product with log2 e is -inf
    ref = dict(i, A=i["A"].clamp(min=-1e30))
    check_scan(i, B, T, D, S, 1, F32, ref)
    if cu is None:
        state = i["init"].clone()
        out = torch.empty(B, D, device=DEV)
        one = lambda n: None if i[n] is None else i[n][:, 0]  # noqa: E731
        kda.kda_selective_scan_step(one("x"), one("delta"), i["A"], one("Bm"), one("Cm"), state,
                                    out, **dict(scan_opt(i), z=one("z")))
        cut = {n: ref[n][:, :1] for n in ("x", "delta", "Bm", "Cm", "z")}
        _, ro, rf = scan_ref(dict(ref, bounds=R.seq_bounds(B, 1, None), **cut))
        near(out, ro)
        near(state, rf)
