"""Edges of the operators around the recurrence on the GPU: every way a batch is
spread (one or two channels a thread, cut or not), offsets beyond 32 bits,
thousands of one-token sequences, values that must not leak, exact cases, the
debug library, two streams at once.
"""
import pytest
import torch

import gated_delta_rule_158_b200 as kda

import layer_ref as R
from test_gpu_layer_ops import (BF16, DEV, F32, Outs, cu_tensor, draw, flat, host, near, ok,
                                scan_inputs, scan_opt, scan_ref)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def scan_forward(i, B, T, D, S, G, ws=None, stream=None):
    n = kda.kda_selective_scan_fwd_workspace_size(B, T, D, S, G, 0 if i["cu"] is None else i["N"])
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if ws is None else ws
    out = torch.full((B, T, D), float("nan"), dtype=i["x"].dtype, device=DEV)
    fin = torch.full((i["N"], D, S), float("nan"), device=DEV)
    kda.kda_selective_scan_fwd(i["x"], i["delta"], i["A"], i["Bm"], i["Cm"], out, ws,
                               init_state=i["init"], cu_seqlens=i["cu"], final_state=fin,
                               stream=stream, **scan_opt(i))
    return out, fin, ws


def scan_backward(i, B, T, D, S, G):
    g = {k: torch.full(s, float("nan"), device=DEV) for k, s in
         dict(dx=(B, T, D), ddelta=(B, T, D), dA=(D, S), dB=(B, T, G, S), dC=(B, T, G, S),
              dD=(D,), dz=(B, T, D), ddelta_bias=(D,), d_init=(i["N"], D, S)).items()}
    n = kda.kda_selective_scan_bwd_workspace_size(B, T, D, S, G, 0 if i["cu"] is None else i["N"])
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    kda.kda_selective_scan_bwd(i["x"], i["delta"], i["A"], i["Bm"], i["Cm"], i["dout"], g, ws,
                               init_state=i["init"], d_final=i["d_final"], cu_seqlens=i["cu"],
                               **scan_opt(i))
    return g, ws


SPREADS = [
    # B, T, D, S, G, cu: two channels a thread without a cut (many channels), ..
    (10, 37, 2048, 16, 1, None),
    (40, 18, 1032, 8, 1, None),
    (3, 35, 3112, 64, 1, None),
    # .. one channel a thread ..
    (4, 41, 2048, 16, 1, None),
    (5, 33, 1024, 32, 2, None),
    (4, 33, 264, 128, 1, None),
    # .. and cut sequences, evenly and with a short last segment
    (1, 513, 264, 64, 1, None),
    (2, 131, 72, 128, 3, None),
    (1, 1100, 24, 8, 1, None),
    # a packed batch whose longest sequence is cut, with empty ones around it
    (1, 1200, 32, 16, 2, [0, 0, 1, 900, 900, 1200, 1200]),
]


@pytest.mark.parametrize("spread", SPREADS)
def test_scan_spreads(spread):
    B, T, D, S, G, cu = spread
    i = scan_inputs((B, T, D, S, G, cu, True, True, True, True, True, False), BF16, seed=31)
    out, fin, ws = scan_forward(i, B, T, D, S, G)
    ok(ws)
    g, ws = scan_backward(i, B, T, D, S, G)
    ok(ws)
    t, ro, rf = scan_ref(i, grad=True)
    near(flat(out), ro, BF16, "out")
    near(fin, rf, what="final")
    ((ro * host(flat(i["dout"]))).sum() + (rf * host(i["d_final"])).sum()).backward()
    for key, src in dict(dx="x", ddelta="delta", dA="A", dB="Bm", dC="Cm", dD="D", dz="z",
                         ddelta_bias="delta_bias", d_init="init").items():
        near(g[key].reshape(t[src].shape), t[src].grad, what=key)


def test_scan_zero_step_leaves_the_state():
    """dt = 0: the state passes through bit for bit, whatever A, x and B are."""
    i = scan_inputs((2, 40, 64, 16, 1, None, False, True, False, False, True, False), F32)
    i["delta"] = torch.zeros_like(i["delta"])
    _, fin, _ = scan_forward(i, 2, 40, 64, 16, 1)
    assert torch.equal(fin, i["init"])
    state = i["init"].clone()
    kda.kda_selective_scan_step(i["x"][:, 0], i["delta"][:, 0], i["A"], i["Bm"][:, 0],
                                i["Cm"][:, 0], state, torch.empty(2, 64, device=DEV),
                                delta_softplus=False)
    assert torch.equal(state, i["init"])


def test_scan_softplus_elementwise():
    """With A = 0 and unit B and C in one state, one token gives y = dt x: the
    softplus itself.  e^-|v| is off by (2 + |v|) 2^-22 (exponential and its
    rounded argument), log1p's polynomial by 2e-7, the additions by 2^-23."""
    v = torch.cat([torch.linspace(-80, 30, 4000), torch.tensor([-1e-30, 0.0, 1e-30, 88.0])])
    D = v.numel() // 8 * 8
    v = v[:D].to(DEV).view(1, 1, D)
    one = torch.zeros(1, 1, 1, 8, device=DEV)
    one[..., 0] = 1
    out = torch.empty(1, 1, D, device=DEV)
    ws = torch.empty(kda.kda_selective_scan_fwd_workspace_size(1, 1, D, 8), dtype=torch.uint8,
                     device=DEV)
    kda.kda_selective_scan_fwd(torch.ones_like(v), v, torch.zeros(D, 8, device=DEV), one, one, out,
                               ws)
    v64 = v.cpu().double()
    ref = v64.clamp(min=0) + torch.log1p(torch.exp(-v64.abs()))
    err = ((out.cpu().double() - ref) / ref).abs()
    assert bool((err <= (2 + v64.abs()) * 2.0 ** -22 + 2e-7 + 2.0 ** -23).all())


def test_values_do_not_leak_between_sequences():
    """NaN and infinities in one packed sequence leave its neighbours alone."""
    cu = [0, 13, 13, 50, 70]
    i = scan_inputs((1, 70, 64, 16, 1, cu, True, True, True, True, True, False), F32, seed=3)
    w = draw(torch.Generator().manual_seed(2), 64, 4)

    def conv():
        out = torch.empty_like(i["x"])
        ws = torch.empty(256, dtype=torch.uint8, device=DEV)
        kda.kda_short_conv_fwd(i["x"], w, out, ws, cu_seqlens=i["cu"])
        return out

    def everything():
        out, fin, _ = scan_forward(i, 1, 70, 64, 16, 1)
        g, _ = scan_backward(i, 1, 70, 64, 16, 1)
        return conv(), out, fin, g

    clean = everything()
    for name in ("x", "Bm", "z"):
        i[name] = i[name].clone()
        i[name][:, 13:50] = float("nan")
        i[name][:, 20] = float("inf")
    i["dout"][:, 13:50] = float("nan")
    dirty = everything()
    for a, b in zip(clean[:2], dirty[:2]):
        assert torch.equal(a[:, :13], b[:, :13]) and torch.equal(a[:, 50:], b[:, 50:])
        assert bool(torch.isnan(b[:, 13:50]).any())
    for n in (0, 1, 3):
        assert torch.equal(clean[2][n], dirty[2][n])
        assert torch.equal(clean[3]["d_init"][n], dirty[3]["d_init"][n])
    for k in ("dx", "ddelta", "dB", "dC", "dz"):
        a, b = clean[3][k], dirty[3][k]
        assert torch.equal(a[:, :13], b[:, :13]) and torch.equal(a[:, 50:], b[:, 50:]), k


def test_norm_rows_stand_alone():
    q = draw(torch.Generator().manual_seed(1), 9, 3, 64)
    k = draw(torch.Generator().manual_seed(2), 9, 2, 64)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    freq = torch.ones(32, device=DEV)
    run = lambda q, k: (kda.kda_qk_norm_fwd(q, k, qo := torch.empty_like(q),  # noqa: E731
                                            ko := torch.empty_like(k), positions=pos,
                                            inv_freq=freq), qo, ko)[1:]
    a = run(q, k)
    q2, k2 = q.clone(), k.clone()
    q2[4, 1] = float("nan")
    k2[7, 0, 5] = float("inf")
    b = run(q2, k2)
    q2[4, 1], k2[7, 0] = q[4, 1], k[7, 0]
    for x, y, at in ((a[0], b[0], (4, 1)), (a[1], b[1], (7, 0))):
        y = y.clone()
        y[at] = x[at]
        assert torch.equal(x, y)


def test_thousands_of_short_sequences():
    """3000 sequences of zero, one or two tokens: each is its own convolution and
    scan, from its own states."""
    N, D, S = 3000, 16, 8
    gen = torch.Generator().manual_seed(12)
    lens = torch.randint(0, 3, (N,), generator=gen)
    cu = [0] + torch.cumsum(lens, 0).tolist()
    T = cu[-1]
    i = scan_inputs((1, T, D, S, 1, cu, True, True, True, True, True, False), F32, seed=4)
    out, fin, ws = scan_forward(i, 1, T, D, S, 1)
    ok(ws)
    _, ro, rf = scan_ref(i)
    near(flat(out), ro)
    near(fin, rf)
    g, ws = scan_backward(i, 1, T, D, S, 1)
    ok(ws)
    empty = torch.tensor([n for n in range(N) if lens[n] == 0], device=DEV)
    assert torch.equal(g["d_init"][empty], i["d_final"][empty])
    w, s0, df = draw(gen, D, 4), draw(gen, N, 3, D), draw(gen, N, 3, D)
    o = Outs()
    y, f = o((1, T, D)), o((N, 3, D))
    kda.kda_short_conv_fwd(i["x"], w, y, ws, init_state=s0, cu_seqlens=i["cu"], final_state=f)
    gc = dict(dx=o((1, T, D)), dweight=o((D, 4)), d_init=o((N, 3, D)))
    wsc = torch.empty(kda.kda_short_conv_bwd_workspace_size(1, T, D, 4, N), dtype=torch.uint8,
                      device=DEV)
    dout = draw(gen, 1, T, D)
    kda.kda_short_conv_bwd(i["x"], w, dout, gc, wsc, init_state=s0, d_final=df,
                           cu_seqlens=i["cu"])
    ok(wsc)
    o.check_guards()
    x64, w64, s64 = host(flat(i["x"]), True), host(w, True), host(s0, True)
    ry, rfin = R.conv(x64, w64, None, s64, i["bounds"], True)
    near(flat(y), ry)
    near(f, rfin)
    ((ry * host(flat(dout))).sum() + (rfin * host(df)).sum()).backward()
    near(flat(gc["dx"]), x64.grad)
    near(gc["dweight"], w64.grad)
    near(gc["d_init"], s64.grad)


# ------------------------------------------------------- offsets beyond 32 bits
def test_conv_beyond_32_bit_offsets():
    """The last sequence of a packed batch of 2.3e9 elements, alone and in place."""
    D, T, tail = 8192, 281000, 700
    x = torch.empty(1, T, D, dtype=BF16, device=DEV).normal_()
    w = torch.randn(D, 4, device=DEV)
    cu = cu_tensor([0, T - tail, T])
    out = torch.empty_like(x)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    fin = torch.empty(2, 3, D, dtype=BF16, device=DEV)
    kda.kda_short_conv_fwd(x, w, out, ws, cu_seqlens=cu, final_state=fin)
    ok(ws)
    alone, last = torch.empty(1, tail, D, dtype=BF16, device=DEV), torch.empty_like(fin[1:])
    kda.kda_short_conv_fwd(x[:, T - tail:], w, alone, ws, final_state=last)
    assert torch.equal(out[:, T - tail:], alone) and torch.equal(fin[1:], last)


def test_scan_beyond_32_bit_offsets():
    D, T, tail, S = 8192, 281000, 300, 8
    x = torch.empty(1, T, D, dtype=BF16, device=DEV).normal_()
    bc = torch.empty(1, T, 1, S, dtype=BF16, device=DEV).normal_()
    A = -torch.rand(D, S, device=DEV)
    out = torch.empty_like(x)
    ws = torch.empty(kda.kda_selective_scan_fwd_workspace_size(1, T, D, S, 1, 2),
                     dtype=torch.uint8, device=DEV)
    fin = torch.empty(2, D, S, device=DEV)
    kda.kda_selective_scan_fwd(x, x, A, bc, bc, out, ws, z=x,
                               cu_seqlens=cu_tensor([0, T - tail, T]), final_state=fin)
    ok(ws)
    alone, last = torch.empty(1, tail, D, dtype=BF16, device=DEV), torch.empty_like(fin[1:])
    part = (x[:, T - tail:], bc[:, T - tail:])
    kda.kda_selective_scan_fwd(part[0], part[0], A, part[1], part[1], alone, ws, z=part[0],
                               final_state=last)
    # segments and channels a thread may differ: sums in another order
    assert R.rel_l2(fin[1:], last) <= 1e-5
    assert R.rel_l2(out[:, T - tail:], alone) <= R.bar(BF16)


def test_norm_beyond_32_bit_offsets():
    tokens, H, d = 290000, 32, 256
    q = torch.empty(tokens, H, d, dtype=BF16, device=DEV).normal_()
    k = q[:, :8].contiguous()
    kda.kda_qk_norm_fwd(q, k, q, k)  # in place
    for t in (q, k):
        n = t[-1000:].float().square().sum(-1)
        # 256 values rounded to bf16 each: the sum of squares within twice half a step
        assert float((n - 1).abs().max()) <= 2 * 2.0 ** -8


# ------------------------------------------------------- debug library, streams
@pytest.mark.parametrize("cu", [None, [0, 0, 31, 31, 400, 600]])
def test_debug_library_is_identical(cu):
    B, T, D, S = (2, 300, 72, 16) if cu is None else (1, 600, 72, 16)
    i = scan_inputs((B, T, D, S, 1, cu, True, True, True, True, True, False), BF16, seed=9)
    w = draw(torch.Generator().manual_seed(5), D, 4)

    def everything():
        out, fin, ws = scan_forward(i, B, T, D, S, 1)
        ok(ws)
        g, ws = scan_backward(i, B, T, D, S, 1)
        ok(ws)
        y = torch.empty_like(i["x"])
        gc = dict(dx=torch.empty(B, T, D, device=DEV), dweight=torch.empty(D, 4, device=DEV))
        ws = torch.empty(kda.kda_short_conv_bwd_workspace_size(B, T, D, 4, 0 if cu is None else 5),
                         dtype=torch.uint8, device=DEV)
        kda.kda_short_conv_fwd(i["x"], w, y, ws, cu_seqlens=i["cu"])
        ok(ws)
        kda.kda_short_conv_bwd(i["x"], w, g["dx"], gc, ws, cu_seqlens=i["cu"])
        ok(ws)
        return [out, fin, y, *g.values(), *gc.values()]

    release = everything()
    kda.select_library(debug=True)
    try:
        debug = everything()
    finally:
        kda.select_library(debug=False)
    for a, b in zip(release, debug):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls on two streams with their own workspaces and outputs do not meet."""
    i = [scan_inputs((2, 500, 256, 16, 1, None, True, True, True, True, True, False), BF16, seed=s)
         for s in (1, 2)]
    alone = [scan_forward(j, 2, 500, 256, 16, 1)[:2] for j in i]
    streams = [torch.cuda.Stream() for _ in i]
    torch.cuda.synchronize()
    both = []
    for _ in range(3):
        for j, s in zip(i, streams):
            with torch.cuda.stream(s):
                both.append(scan_forward(j, 2, 500, 256, 16, 1)[:2])
    torch.cuda.synchronize()
    for k, pair in enumerate(both):
        for a, b in zip(pair, alone[k % 2]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("spread", [
    # a packed batch is cut only where a sequence has more than 512 tokens (with
    # few channels): the longest just at the limit, just beyond it, and beyond it
    # in the last and in a single sequence
    (1, 1200, 32, 16, 2, [0, 512, 600, 600, 1112, 1200]),
    (1, 1200, 32, 16, 2, [0, 513, 600, 600, 1112, 1200]),
    (1, 1200, 40, 8, 1, [0, 1, 65, 130, 1200]),
    (1, 545, 264, 128, 1, [0, 545]),
    (1, 512, 264, 32, 1, [0, 512]),
])
def test_packed_batches_around_the_cut(spread):
    test_scan_spreads(spread)


@pytest.mark.parametrize("kind", ["conv", "scan"])
def test_steps_of_many_sequences(kind):
    """Steps on both sides of the size from which a thread takes four sequences,
    with and without a remainder: bit-identical to the sequences one by one."""
    gen = torch.Generator().manual_seed(3)
    for N in (1, 31, 45, 122):
        if kind == "conv":
            D, Wd = 5000, 4
            x, w, b = draw(gen, N, D, dtype=BF16), draw(gen, D, Wd, scale=0.5), draw(gen, D)
            state = draw(gen, N, Wd - 1, D, dtype=BF16)
            one, out, ref = state.clone(), torch.empty_like(x), torch.empty_like(x)
            kda.kda_short_conv_step(x, w, state, out, bias=b)
            for n in range(N):
                kda.kda_short_conv_step(x[n:n + 1], w, one[n:n + 1], ref[n:n + 1], bias=b)
        else:
            D, S = 1504, 32
            x, delta, z = (draw(gen, N, D, dtype=BF16) for _ in range(3))
            A = -torch.rand(D, S, generator=gen).to(DEV) * S
            Bm, Cm = (draw(gen, N, 1, S, dtype=BF16) for _ in range(2))
            state = draw(gen, N, D, S)
            one, out, ref = state.clone(), torch.empty_like(x), torch.empty_like(x)
            kda.kda_selective_scan_step(x, delta, A, Bm, Cm, state, out, z=z)
            for n in range(N):
                k = slice(n, n + 1)
                kda.kda_selective_scan_step(x[k], delta[k], A, Bm[k], Cm[k], one[k], ref[k],
                                            z=z[k])
        assert torch.equal(state, one)
        # the scan's outputs are summed over a channel's lanes in another order
        if kind == "conv":
            assert torch.equal(out, ref)
        else:
            near(out, host(ref), BF16)
