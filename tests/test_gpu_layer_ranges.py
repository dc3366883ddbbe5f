"""The operators around the recurrence over the ranges of their inputs on the
GPU, against the fp64 references."""
import pytest
import torch

import gated_delta_rule_158_b200 as kda

import layer_ref as R
from test_gpu_layer_edges import scan_backward, scan_forward
from test_gpu_layer_ops import (BF16, DEV, F32, draw, flat, host, near, ok, scan_inputs, scan_opt,
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


# ------------------------------------------------------------------- norms
def norm_call(T, Hq, Hk, d, rot, dtype, seed=6):
    gen = torch.Generator().manual_seed(seed)
    t = dict(q=draw(gen, T, Hq, d, dtype=dtype), k=draw(gen, T, Hk, d, dtype=dtype),
             dq=draw(gen, T, Hq, d), dk=draw(gen, T, Hk, d))
    opt = dict(q_weight=0.5 + torch.rand(d, generator=gen).to(DEV),
               k_weight=0.5 + torch.rand(d, generator=gen).to(DEV), mode=kda.KDA_NORM_RMS)
    if rot:
        opt.update(positions=torch.arange(T, dtype=torch.int32, device=DEV),
                   inv_freq=torch.rand(rot // 2, generator=gen).to(DEV))
    e = lambda x, dt=F32: torch.full(x.shape, float("nan"), dtype=dt, device=DEV)  # noqa: E731
    out = dict(q=e(t["q"], dtype), k=e(t["k"], dtype))
    g = dict(dq=e(t["q"]), dk=e(t["k"]), dq_weight=e(opt["q_weight"]), dk_weight=e(opt["k_weight"]))
    ws = torch.empty(kda.kda_qk_norm_bwd_workspace_size(T, Hq, Hk, d), dtype=torch.uint8,
                     device=DEV)
    fwd = lambda: kda.kda_qk_norm_fwd(t["q"], t["k"], out["q"], out["k"], **opt)  # noqa: E731
    bwd = lambda: kda.kda_qk_norm_bwd(t["q"], t["k"], t["dq"], t["dk"], g, ws, **opt)  # noqa: E731
    return t, opt, out, g, fwd, bwd


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,Hq,Hk,d,rot", [
    # few heads: tiles of many tokens, of all sizes around a tile for every block
    (9473, 1, 1, 32, 0), (9473, 1, 1, 32, 32), (2401, 1, 2, 64, 0), (1777, 1, 1, 8, 0),
    (593, 3, 1, 96, 96), (297, 1, 1, 32, 16),
    # more heads than fit beside one another, and as many
    (1201, 8, 1, 128, 0), (1185, 9, 8, 128, 128), (700, 5, 3, 256, 64), (1185, 40, 24, 16, 16),
])
def test_norm_tiles(T, Hq, Hk, d, rot, dtype):
    t, opt, out, g, fwd, bwd = norm_call(T, Hq, Hk, d, rot, dtype)
    fwd()
    bwd()
    freq = opt["inv_freq"].cpu() if rot else None
    for n in ("q", "k"):
        x, w = host(t[n], True), host(opt[n + "_weight"], True)
        y = R.norm(x, w, torch.arange(T), freq, False, False, 1e-6)
        near(out[n], y, dtype, n)
        y.backward(host(t["d" + n]))
        near(g["d" + n], x.grad, what="d" + n)
        near(g[f"d{n}_weight"], w.grad, what=n + " weight")


def microseconds(f):
    for _ in range(3):
        f()
    times = []
    for _ in range(30):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return min(times)


@pytest.mark.parametrize("rot", [0, 32])
def test_norm_of_fewer_tokens_takes_no_longer(rot):
    """16,384 tokens of two short heads against 40,000: less than half the work.
    (With one token a step and block, most lanes idle, they took three times as long.)"""
    few = norm_call(16384, 1, 1, 32, rot, BF16)[-2:]
    many = norm_call(40000, 1, 1, 32, rot, BF16)[-2:]
    for a, b in zip(few, many):
        assert microseconds(a) <= 1.5 * microseconds(b)


# ------------------------------------------------- one long sequence, few channels
@pytest.mark.parametrize("cu", [None, [0, 11000, 12000]])
def test_scan_of_a_long_sequence(cu):
    """More tokens than a sequence's segments times the shortest segment: the
    segments are longer, in dense and in packed batches."""
    B, T, D, S = 1, 12000, 8, 8
    i = scan_inputs((B, T, D, S, 1, cu, True, True, True, True, True, False), F32, seed=17)
    check_scan(i, B, T, D, S, 1, F32)


@pytest.mark.parametrize("packed", [False, True])
def test_scan_gradients_of_four_times_the_tokens(packed):
    """65,536 tokens of 64 channels against 16,384.  (Cut into 1024 segments, whose
    combination is one chain, they took 3.8 times as long.)"""
    def backward(T, D=64, S=16):
        gen = torch.Generator(device=DEV).manual_seed(1)
        n = lambda *s: torch.randn(s, generator=gen, device=DEV).to(BF16)  # noqa: E731
        x, bc = n(1, T, D), n(1, T, 1, S)
        A = -0.1 - torch.rand(D, S, generator=gen, device=DEV)
        e = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
        g = dict(dx=e(1, T, D), ddelta=e(1, T, D), dA=e(D, S), dB=e(1, T, 1, S), dC=e(1, T, 1, S))
        cu = torch.tensor([0, T], dtype=torch.int32, device=DEV) if packed else None
        ws = torch.empty(kda.kda_selective_scan_bwd_workspace_size(1, T, D, S, 1, int(packed)),
                         dtype=torch.uint8, device=DEV)
        return lambda: kda.kda_selective_scan_bwd(x, x, A, bc, bc, x, g, ws, cu_seqlens=cu)
    assert microseconds(backward(65536)) <= 3 * microseconds(backward(16384))


# ----------------------------------------------------- packed: many sequences
def lengths(N, seed=5, most=6):
    gen = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, most + 1, (N,), generator=gen)
    return [0] + torch.cumsum(lens, 0).tolist()


@pytest.mark.parametrize("N", [511, 512, 513])
def test_scan_around_the_last_ordered_batch(N):
    cu = lengths(N)
    i = scan_inputs((1, cu[-1], 8, 8, 1, cu, True, True, True, True, True, False), F32, seed=N)
    check_scan(i, 1, cu[-1], 8, 8, 1, F32)


def test_scan_plan_of_many_sequences():
    """2048 sequences of eight tokens against 2049.  (Ordered by N^2 comparisons, the
    2048 took 3.6 times as long.)"""
    def forward(N, T=16384, D=64, S=16):
        gen = torch.Generator(device=DEV).manual_seed(1)
        n = lambda *s: torch.randn(s, generator=gen, device=DEV).to(BF16)  # noqa: E731
        x, bc = n(1, T, D), n(1, T, 1, S)
        A, out = -torch.ones(D, S, device=DEV), torch.empty(1, T, D, dtype=BF16, device=DEV)
        cu = (torch.arange(N + 1, device=DEV) * T // N).to(torch.int32)
        ws = torch.empty(kda.kda_selective_scan_fwd_workspace_size(1, T, D, S, 1, N),
                         dtype=torch.uint8, device=DEV)
        return lambda: kda.kda_selective_scan_fwd(x, x, A, bc, bc, out, ws, cu_seqlens=cu)
    assert microseconds(forward(2048)) <= 1.5 * microseconds(forward(2049))
