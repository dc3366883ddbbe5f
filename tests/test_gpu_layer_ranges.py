"""The operators around the recurrence over the ranges of their inputs on the
GPU, against the fp64 references."""
import pytest
import torch

import gated_delta_rule_158_b200 as kda

import layer_ref as R
from test_gpu_layer_edges import SPREADS, scan_backward, scan_forward
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


# --------------------------------------------------------------- types, values
@pytest.mark.parametrize("spread", SPREADS)
def test_scan_spreads_fp32(spread):
    B, T, D, S, G, cu = spread
    i = scan_inputs((B, T, D, S, G, cu, True, True, True, True, True, False), F32, seed=33)
    check_scan(i, B, T, D, S, G, F32)


def test_softplus_of_special_values():
    """One token, A = 0, unit B and C in one state: y = softplus(v) itself, by the
    prompt's kernel and by the step's.  e^-|v| is off by (2 + |v|) 2^-22 (the
    exponential and its rounded argument), the polynomial by 1.5e-7, the additions
    by 2^-23.  Below -87.3 e^v is no normal fp32 number, and 0."""
    v = torch.tensor([-1e-30, 0.0, 1e-30, 88.0, 1e-6, -1e-6, 0.5, -0.5, -5.0, 5.0, -16.0, 16.0,
                      -17.5, -80.0, 1000.0, -1000.0], device=DEV)
    D = v.numel()
    one = torch.zeros(1, 1, 1, 8, device=DEV)
    one[..., 0] = 1
    A, x = torch.zeros(D, 8, device=DEV), torch.ones(1, 1, D, device=DEV)
    out, step = torch.empty(1, 1, D, device=DEV), torch.empty(1, D, device=DEV)
    ws = torch.empty(kda.kda_selective_scan_fwd_workspace_size(1, 1, D, 8), dtype=torch.uint8,
                     device=DEV)
    kda.kda_selective_scan_fwd(x, v.view(1, 1, D), A, one, one, out, ws)
    kda.kda_selective_scan_step(x[0], v.view(1, D), A, one[0], one[0],
                                torch.zeros(1, D, 8, device=DEV), step)
    v64 = v.cpu().double()
    ref = v64.clamp(min=0) + torch.log1p(torch.exp(-v64.abs()))
    ref[-1] = 0.0
    bar = ref * ((2 + v64.abs().clamp(max=100)) * 2.0 ** -22 + 1.5e-7 + 2.0 ** -23)
    for y in (out, step):
        y = y.cpu().double().view(-1)
        assert bool(((y - ref).abs() <= bar).all()), y - ref


# ------------------------------------------------- steps of many sequences, fp64
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S,D,G,N", [(16, 1032, 1, 78), (16, 1024, 4, 77), (32, 512, 2, 75),
                                     (64, 264, 1, 75), (128, 192, 3, 50)])
def test_scan_step_of_many_sequences(S, D, G, N, dtype):
    """Four sequences a thread (ceil(N / 4) D S / 4 threads, above 148 x 512), the
    last group not full, with all optional inputs."""
    assert (N + 3) // 4 * D * S // 4 >= 148 * 512 and N % 4
    i = scan_inputs((N, 1, D, S, G, None, True, True, True, True, True, True), dtype, seed=51)
    state, out = i["init"].clone(), torch.full((N, D), float("nan"), dtype=dtype, device=DEV)
    one = lambda n: i[n][:, 0]  # noqa: E731
    kda.kda_selective_scan_step(one("x"), one("delta"), i["A"], one("Bm"), one("Cm"), state, out,
                                **dict(scan_opt(i), z=one("z")))
    _, ro, rf = scan_ref(i)
    near(out, ro, dtype)
    near(state, rf)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Wd,silu,bias", [(2, True, True), (3, False, True), (4, False, False),
                                          (4, True, True)])
def test_conv_step_of_many_sequences(Wd, silu, bias, dtype):
    """Four sequences a thread (ceil(N / 4) D / 4 threads, above 148 x 256)."""
    N, D = 146, 4104
    assert (N + 3) // 4 * D // 4 >= 148 * 256 and N % 4
    gen = torch.Generator().manual_seed(52)
    x = draw(gen, N, D, dtype=dtype)
    w, b = draw(gen, D, Wd, scale=0.5), draw(gen, D) if bias else None
    state = draw(gen, N, Wd - 1, D, dtype=dtype)
    rows = torch.cat([host(state), host(x)[:, None]], 1)
    out = torch.full((N, D), float("nan"), dtype=dtype, device=DEV)
    kda.kda_short_conv_step(x, w, state, out, bias=b,
                            activation=kda.KDA_ACT_SILU if silu else kda.KDA_ACT_NONE)
    p = (rows * host(w).t()).sum(1) + (host(b) if bias else 0)
    near(out, p * torch.sigmoid(p) if silu else p, dtype)
    assert torch.equal(host(state), rows[:, 1:])


# ------------------------------------------- gradients at offsets beyond 32 bits
# the last sequence of a packed batch of more than 2^31 elements; the cotangents
# in front of it are zero, so that the sums over all tokens are its own too
BIG_T, BIG_D, TAIL = 263000, 8192, 300
BIG_CU = [0, BIG_T - TAIL, BIG_T]


def big(dtype=BF16):
    torch.cuda.empty_cache()
    return torch.empty(1, BIG_T, BIG_D, dtype=dtype, device=DEV)


def last(t):
    return t[:, BIG_T - TAIL:]


def same(whole, alone, what):
    # the strips and segments differ: other orders of the same sums
    assert R.rel_l2(whole, alone) <= 1e-5, (what, R.rel_l2(whole, alone))


def test_conv_gradients_beyond_32_bit_offsets():
    x = big().normal_()
    dout = big(F32).zero_()
    last(dout).normal_()
    w = torch.randn(BIG_D, 4, device=DEV)
    g = dict(dx=big(F32), dweight=torch.empty_like(w), dbias=torch.empty(BIG_D, device=DEV),
             d_init=torch.empty(2, 3, BIG_D, device=DEV))
    ws = torch.empty(kda.kda_short_conv_bwd_workspace_size(1, BIG_T, BIG_D, 4, 2),
                     dtype=torch.uint8, device=DEV)
    b = torch.randn(BIG_D, device=DEV)
    kda.kda_short_conv_bwd(x, w, dout, g, ws, bias=b,
                           cu_seqlens=torch.tensor(BIG_CU, dtype=torch.int32, device=DEV))
    ok(ws)
    a = dict(dx=torch.empty(1, TAIL, BIG_D, device=DEV), dweight=torch.empty_like(w),
             dbias=torch.empty_like(b), d_init=torch.empty(1, 3, BIG_D, device=DEV))
    kda.kda_short_conv_bwd(last(x), w, last(dout), a, ws, bias=b)
    same(last(g["dx"]), a["dx"], "dx")
    assert not bool(g["dx"][:, BIG_T - TAIL - 1000:BIG_T - TAIL].any())
    for k in ("dweight", "dbias"):
        same(g[k], a[k], k)
    same(g["d_init"][1:], a["d_init"], "d_init")


def test_scan_gradients_beyond_32_bit_offsets():
    S = 8
    x = big().normal_()
    dout = big().zero_()
    last(dout).normal_()
    bc = torch.randn(1, BIG_T, 1, S, device=DEV).to(BF16)
    A = -torch.rand(BIG_D, S, device=DEV) - 0.1
    f32 = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    g = dict(dx=big(F32), ddelta=big(F32), dz=big(F32), dA=f32(BIG_D, S),
             dB=f32(1, BIG_T, 1, S), dC=f32(1, BIG_T, 1, S), dD=f32(BIG_D),
             ddelta_bias=f32(BIG_D), d_init=f32(2, BIG_D, S))
    ws = torch.empty(kda.kda_selective_scan_bwd_workspace_size(1, BIG_T, BIG_D, S, 1, 2),
                     dtype=torch.uint8, device=DEV)
    kda.kda_selective_scan_bwd(x, x, A, bc, bc, dout, g, ws, z=x,
                               cu_seqlens=torch.tensor(BIG_CU, dtype=torch.int32, device=DEV))
    ok(ws)
    a = {k: f32(1, TAIL, *g[k].shape[2:]) for k in ("dx", "ddelta", "dz", "dB", "dC")}
    a.update({k: torch.empty_like(g[k]) for k in ("dA", "dD", "ddelta_bias")},
             d_init=f32(1, BIG_D, S))
    part, mix = last(x), last(bc)
    kda.kda_selective_scan_bwd(part, part, A, mix, mix, last(dout), a, ws, z=part)
    for k in ("dx", "ddelta", "dz", "dB", "dC"):
        same(last(g[k]), a[k], k)
    for k in ("dA", "dD", "ddelta_bias"):
        same(g[k], a[k], k)
    same(g["d_init"][1:], a["d_init"], "d_init")


def test_norm_gradients_beyond_32_bit_offsets():
    tokens, H, Hk, d, tail = 263000, 32, 2, 256, 300
    torch.cuda.empty_cache()
    q = torch.empty(tokens, H, d, dtype=BF16, device=DEV).normal_()
    k = q[:, :Hk].contiguous()
    dq, dk = torch.zeros(tokens, H, d, device=DEV), torch.zeros(tokens, Hk, d, device=DEV)
    dq[-tail:].normal_()
    dk[-tail:].normal_()
    w = 0.5 + torch.rand(d, device=DEV)
    pos = torch.arange(tokens, dtype=torch.int32, device=DEV)
    opt = dict(q_weight=w, k_weight=w, inv_freq=torch.rand(32, device=DEV))
    e = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    a = dict(dq=e(tail, H, d), dk=e(tail, Hk, d), dq_weight=e(d), dk_weight=e(d))
    ws = torch.empty(kda.kda_qk_norm_bwd_workspace_size(tokens, H, Hk, d), dtype=torch.uint8,
                     device=DEV)
    kda.kda_qk_norm_bwd(q[-tail:], k[-tail:], dq[-tail:], dk[-tail:], a, ws,
                        positions=pos[-tail:].clone(), **opt)
    g = dict(dq=dq, dk=dk, dq_weight=e(d), dk_weight=e(d))  # over the cotangents
    kda.kda_qk_norm_bwd(q, k, dq, dk, g, ws, positions=pos, **opt)
    for n in ("dq", "dk"):
        same(g[n][-tail:], a[n], n)
        assert not bool(g[n][-tail - 1000:-tail].any())
        same(g[n + "_weight"], a[n + "_weight"], n + " weight")


# ----------------------------------------------------------- gradients in parts
def test_scan_gradients_in_parts():
    """A sequence's gradients from its last part to its first, the states passed
    forward and the state gradients back: those of the whole."""
    B, T, D, S, cut = 2, 130, 40, 16, 77
    i = scan_inputs((B, T, D, S, 1, None, True, True, True, True, True, False), F32, seed=61)
    whole, ws = scan_backward(i, B, T, D, S, 1)
    ok(ws)
    part = {}
    state, d_state = i["init"], i["d_final"]
    for a, b in ((0, cut), (cut, T)):
        p = dict(i, init=state)
        p.update({n: i[n][:, a:b].contiguous() for n in ("x", "delta", "Bm", "Cm", "z", "dout")})
        part[a] = p
        _, state, _ = scan_forward(p, B, b - a, D, S, 1)
    grads = {}
    for a, b in ((cut, T), (0, cut)):
        g, ws = scan_backward(dict(part[a], d_final=d_state), B, b - a, D, S, 1)
        ok(ws)
        grads[a], d_state = g, g["d_init"]
    for n in ("dx", "ddelta", "dB", "dC", "dz"):
        same(torch.cat([grads[0][n], grads[cut][n]], 1), whole[n], n)
    for n in ("dA", "dD", "ddelta_bias"):
        same(grads[0][n] + grads[cut][n], whole[n], n)
    same(grads[0]["d_init"], whole["d_init"], "d_init")


# ------------------------------------------------------------- sigmoid, element by element
def test_silu_and_gate_elementwise():
    """fp32 callers' SiLU and gate: the sigmoid within (3 + |x|) 2^-22 of itself, and
    a rounding (2^-24) for each product behind it.  A tap of one and zeros make the
    convolution x sigmoid(x); B = C = 0 and a skip of one make the scan z sigmoid(z)."""
    v = torch.cat([torch.linspace(-80, 80, 4089), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-4,
                                                                -1e-4, 20.0])]).to(DEV)
    D = v.numel()
    assert D % 8 == 0
    w = torch.zeros(D, 2, device=DEV)
    w[:, 1] = 1
    outs = [torch.empty(1, 1, D, device=DEV) for _ in range(4)]
    ws = torch.empty(kda.kda_selective_scan_fwd_workspace_size(1, 1, D, 8), dtype=torch.uint8,
                     device=DEV)
    kda.kda_short_conv_fwd(v.view(1, 1, D), w, outs[0], ws)
    kda.kda_short_conv_step(v.view(1, D), w, torch.zeros(1, 1, D, device=DEV), outs[1][0])
    one, none, A = torch.ones(1, 1, D, device=DEV), torch.zeros(1, 1, 1, 8, device=DEV), \
        torch.zeros(D, 8, device=DEV)
    opt = dict(D=one.view(D), z=v.view(1, 1, D))
    kda.kda_selective_scan_fwd(one, one, A, none, none, outs[2], ws, **opt)
    opt["z"] = v.view(1, D)
    kda.kda_selective_scan_step(one[0], one[0], A, none[0], none[0],
                                torch.zeros(1, D, 8, device=DEV), outs[3][0], **opt)
    x = v.cpu().double()
    ref = x * torch.sigmoid(x)
    bar = ref.abs() * ((3 + x.abs()) * 2.0 ** -22 + 2 * 2.0 ** -24)
    for out in outs:
        err = (out.view(D).cpu().double() - ref).abs()
        assert bool((err <= bar).all()), float((err / ref.abs()).nan_to_num().max())


def test_scan_nan_in_a_rate_stays_in_its_channel():
    i = scan_inputs((2, 33, 40, 16, 1, None, True, True, True, True, True, False), F32, seed=41)
    clean = scan_forward(i, 2, 33, 40, 16, 1)[:2]
    i["A"][7, 3] = float("nan")
    out, fin, _ = scan_forward(i, 2, 33, 40, 16, 1)
    assert bool(torch.isnan(out[..., 7]).all()) and bool(torch.isnan(fin[:, 7, 3]).all())
    out[..., 7], fin[:, 7, 3] = clean[0][..., 7], clean[1][:, 7, 3]
    assert torch.equal(out, clean[0]) and torch.equal(fin, clean[1])
