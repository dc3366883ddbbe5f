"""The operators around the recurrence on the GPU against their fp64
references: the short convolution, the selective scan, the norms with
rotation -- prompts, single tokens and gradients; odd sizes, packed batches
with empty sequences, strided rows, graphs, streams, malformed offsets.

Outputs start as NaN between guard values, so that an element not written and
a store outside are both seen.
"""
import pytest
import torch

import gated_delta_rule_158_b200 as kda
from gated_delta_rule_158_b200 import workloads as W

import layer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


GUARD = 64


class Outs:
    """Output tensors inside guarded, NaN-filled buffers."""

    def __init__(self):
        self.bufs = []

    def __call__(self, shape, dtype=F32):
        n = 1
        for s in shape:
            n *= s
        buf = torch.full((n + 2 * GUARD,), 77.0, dtype=dtype, device=DEV)
        view = buf[GUARD:GUARD + n]
        view.fill_(float("nan"))
        self.bufs.append(buf)
        return view.view(shape)

    def check_guards(self):
        for b in self.bufs:
            assert bool((b[:GUARD] == 77).all()) and bool((b[-GUARD:] == 77).all())


def draw(gen, *shape, scale=1.0, dtype=F32):
    return (torch.randn(shape, generator=gen) * scale).to(dtype).to(DEV)


def rows_of(t, wide, gen):
    """The same values as slices of wider rows, 16 elements in."""
    if not wide:
        return t
    lead, width = t.shape[:-1], t.shape[-1]
    buf = torch.full((*lead, width + 32), 1e30, dtype=t.dtype, device=DEV)
    buf[..., 16:16 + width] = t
    return buf[..., 16:16 + width]


def host(t, grad=False):
    if t is None:
        return None
    return t.detach().to("cpu", R.F64).requires_grad_(grad)


def flat(t):
    return None if t is None else t.reshape(-1, *t.shape[2:])


def cu_tensor(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)


def near(got, ref, dtype=F32, what=""):
    assert bool(torch.isfinite(got).all()), what
    assert got.shape == ref.shape, what
    assert R.rel_l2(got, ref) <= R.bar(dtype), (what, R.rel_l2(got, ref))


def ok(ws):
    st, _ = kda.kda_get_device_status(ws)
    assert st == kda.KDA_OK, kda.kda_status_string(st)


RAGGED = [0, 3, 3, 4, 41, 41, 73, 74, 76]  # empty, one-token, shorter than the taps

# ------------------------------------------------------------ short convolution
CONV_CASES = [
    # B, T, D, W, cu, silu, bias, state, wide
    (1, 1, 8, 4, None, True, True, True, False),
    (2, 2, 24, 4, None, True, False, True, True),
    (3, 37, 40, 3, None, False, True, False, False),
    (1, 131, 264, 2, None, True, True, True, True),
    (2, 200, 2056, 4, None, True, True, False, False),
    (1, 76, 72, 4, RAGGED, True, True, True, True),
    (1, 76, 72, 3, RAGGED, True, False, False, False),
    (1, 76, 1032, 2, RAGGED, False, True, True, False),
]


def conv_inputs(case, dtype, seed=1):
    B, T, D, Wd, cu, silu, bias, state, wide = case
    gen = torch.Generator().manual_seed(seed)
    N = B if cu is None else len(cu) - 1
    i = dict(x=rows_of(draw(gen, B, T, D, dtype=dtype), wide, gen),
             weight=draw(gen, D, Wd, scale=0.5), bias=draw(gen, D) if bias else None,
             init=draw(gen, N, Wd - 1, D, dtype=dtype) if state else None,
             dout=draw(gen, B, T, D), d_final=draw(gen, N, Wd - 1, D) if state else None,
             act=kda.KDA_ACT_SILU if silu else kda.KDA_ACT_NONE, cu=cu_tensor(cu), N=N,
             bounds=R.seq_bounds(B, T, cu))
    return i


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CONV_CASES)
def test_conv_forward(case, dtype):
    B, T, D, Wd, cu, silu, *_ = case
    i = conv_inputs(case, dtype)
    o = Outs()
    out, fin = o((B, T, D), dtype), o((i["N"], Wd - 1, D), dtype)
    ws = torch.full((256,), 255, dtype=torch.uint8, device=DEV)
    kda.kda_short_conv_fwd(i["x"], i["weight"], out, ws, bias=i["bias"], init_state=i["init"],
                           cu_seqlens=i["cu"], final_state=fin, activation=i["act"])
    ok(ws)
    o.check_guards()
    ro, rf = R.conv(host(flat(i["x"])), host(i["weight"]), host(i["bias"]), host(i["init"]),
                    i["bounds"], silu)
    near(flat(out), ro, dtype)
    assert torch.equal(host(fin), rf)  # rows pass through unchanged


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CONV_CASES)
def test_conv_gradients(case, dtype):
    B, T, D, Wd, cu, silu, bias, state, _ = case
    i = conv_inputs(case, dtype, seed=2)
    o = Outs()
    g = dict(dx=o((B, T, D)), dweight=o((D, Wd)))
    if bias:
        g["dbias"] = o((D,))
    if state:
        g["d_init"] = o((i["N"], Wd - 1, D))
    n = kda.kda_short_conv_bwd_workspace_size(B, T, D, Wd, 0 if cu is None else i["N"])
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    kda.kda_short_conv_bwd(i["x"], i["weight"], i["dout"], g, ws, bias=i["bias"],
                           init_state=i["init"], d_final=i["d_final"], cu_seqlens=i["cu"],
                           activation=i["act"])
    ok(ws)
    o.check_guards()
    x, w, b, s0 = (host(t, True) if t is not None else None
                   for t in (flat(i["x"]), i["weight"], i["bias"], i["init"]))
    ro, rf = R.conv(x, w, b, s0, i["bounds"], silu)
    loss = (ro * host(flat(i["dout"]))).sum()
    if state:
        loss = loss + (rf * host(i["d_final"])).sum()
    loss.backward()
    near(flat(g["dx"]), x.grad, what="dx")
    near(g["dweight"], w.grad, what="dweight")
    if bias:
        near(g["dbias"], b.grad, what="dbias")
    if state:
        near(g["d_init"], s0.grad, what="d_init")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,D,Wd", [(1, 8, 4), (3, 136, 3), (7, 520, 2), (33, 4096, 4)])
def test_conv_step_continues_a_prompt(N, D, Wd, dtype):
    """The prompt's final state and single tokens give the longer prompt's rows."""
    gen = torch.Generator().manual_seed(7)
    T, K = 5, 4
    x = draw(gen, N, T + K, D, dtype=dtype)
    w, b = draw(gen, D, Wd, scale=0.5), draw(gen, D)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    whole = torch.empty(N, T + K, D, dtype=dtype, device=DEV)
    end = torch.empty(N, Wd - 1, D, dtype=dtype, device=DEV)
    kda.kda_short_conv_fwd(x, w, whole, ws, bias=b, final_state=end)
    o = Outs()
    state, out = o((N, Wd - 1, D), dtype), o((N, D), dtype)
    kda.kda_short_conv_fwd(x[:, :T].contiguous(), w, torch.empty_like(whole[:, :T]).contiguous(),
                           ws, bias=b, final_state=state)
    for k in range(K):
        kda.kda_short_conv_step(x[:, T + k], w, state, out, bias=b)  # rows T + K apart
        assert torch.equal(out, whole[:, T + k])
    assert torch.equal(state, end)
    o.check_guards()


# ------------------------------------------------------------ selective scan
SCAN_CASES = [
    # B, T, D, S, G, cu, gate, skip, bias, softplus, state, wide
    (1, 1, 8, 16, 1, None, True, True, True, True, True, False),
    (2, 33, 40, 8, 1, None, True, True, True, True, False, True),
    (1, 70, 64, 16, 2, None, True, True, True, True, True, True),
    (2, 31, 128, 32, 4, None, False, True, True, True, True, False),
    (1, 65, 72, 64, 1, None, True, False, True, True, True, False),
    (2, 17, 24, 128, 1, None, True, True, False, True, True, False),
    (1, 76, 104, 16, 1, RAGGED, True, True, True, True, True, True),
    (1, 76, 64, 64, 2, RAGGED, False, False, False, False, False, False),
    (1, 76, 48, 8, 1, RAGGED, True, True, True, True, True, False),
    (1, 76, 32, 128, 1, RAGGED, True, True, True, True, False, False),
    # long enough to be cut into segments
    (1, 700, 16, 16, 1, None, True, True, True, True, True, False),
    (1, 900, 40, 32, 1, [0, 0, 520, 523, 900], True, True, True, True, True, False),
]


def scan_inputs(case, dtype, seed=1):
    """Step sizes log-uniform in [0.01, 0.5] behind the softplus, decays 1..S:
    a state remembers 100 tokens at most, so the decays' 2^-22 errors add up to
    a few 1e-6 of it."""
    B, T, D, S, G, cu, gate, skip, bias, softplus, state, wide = case
    gen = torch.Generator().manual_seed(seed)
    N = B if cu is None else len(cu) - 1
    step = R.log_uniform(gen, D, 0.01, 0.5)
    raw = torch.log(torch.expm1(step)) if softplus else step
    if bias:
        delta = draw(gen, B, T, D, scale=0.5 if softplus else 0.0, dtype=dtype)
        db = raw.float().to(DEV)
    else:
        delta, db = (raw + 0.02 * torch.randn(B, T, D, generator=gen)).to(dtype).to(DEV), None
    A = -(torch.arange(1, S + 1) * (0.7 + 0.6 * torch.rand(D, S, generator=gen))).float().to(DEV)
    r = lambda t: rows_of(t, wide, gen)  # noqa: E731
    Bm, Cm = (draw(gen, B, T, G * S, dtype=dtype) for _ in range(2))
    Bm, Cm = (r(t).unflatten(-1, (G, S)) for t in (Bm, Cm))
    i = dict(x=r(draw(gen, B, T, D, dtype=dtype)), delta=r(delta), A=A, Bm=Bm, Cm=Cm,
             D=draw(gen, D) if skip else None,
             z=r(draw(gen, B, T, D, dtype=dtype)) if gate else None, delta_bias=db,
             init=draw(gen, N, D, S) if state else None,
             dout=draw(gen, B, T, D, dtype=dtype), d_final=draw(gen, N, D, S) if state else None,
             cu=cu_tensor(cu), N=N, bounds=R.seq_bounds(B, T, cu), softplus=softplus)
    return i


def scan_ref(i, grad=False):
    t = {k: host(flat(i[k]) if k in ("x", "delta", "Bm", "Cm", "z") else i[k], grad)
         if i[k] is not None else None
         for k in ("x", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias", "init")}
    out, fin = R.scan(t["x"], t["delta"], t["A"], t["Bm"], t["Cm"], t["D"], t["z"],
                      t["delta_bias"], i["softplus"], t["init"], i["bounds"])
    return t, out, fin


def scan_opt(i):
    return dict(D=i["D"], z=i["z"], delta_bias=i["delta_bias"], delta_softplus=i["softplus"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", SCAN_CASES)
def test_scan_forward(case, dtype):
    B, T, D, S, G, cu = case[:6]
    i = scan_inputs(case, dtype)
    o = Outs()
    out, fin = o((B, T, D), dtype), o((i["N"], D, S))
    n = kda.kda_selective_scan_fwd_workspace_size(B, T, D, S, G, 0 if cu is None else i["N"])
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    kda.kda_selective_scan_fwd(i["x"], i["delta"], i["A"], i["Bm"], i["Cm"], out, ws,
                               init_state=i["init"], cu_seqlens=i["cu"], final_state=fin,
                               **scan_opt(i))
    ok(ws)
    o.check_guards()
    _, ro, rf = scan_ref(i)
    near(flat(out), ro, dtype, "out")
    near(fin, rf, what="final")
    if i["init"] is not None:  # the state in place
        state, again = i["init"].clone(), o((B, T, D), dtype)
        kda.kda_selective_scan_fwd(i["x"], i["delta"], i["A"], i["Bm"], i["Cm"], again, ws,
                                   init_state=state, cu_seqlens=i["cu"], final_state=state,
                                   **scan_opt(i))
        assert torch.equal(state, fin) and torch.equal(again, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", SCAN_CASES)
def test_scan_gradients(case, dtype):
    B, T, D, S, G, cu = case[:6]
    i = scan_inputs(case, dtype, seed=2)
    o = Outs()
    g = dict(dx=o((B, T, D)), ddelta=o((B, T, D)), dA=o((D, S)), dB=o((B, T, G, S)),
             dC=o((B, T, G, S)))
    names = dict(dx="x", ddelta="delta", dA="A", dB="Bm", dC="Cm")
    for key, src, shape in (("dD", "D", (D,)), ("dz", "z", (B, T, D)),
                            ("ddelta_bias", "delta_bias", (D,)), ("d_init", "init", (i["N"], D, S))):
        if i[src] is not None:
            g[key] = o(shape)
            names[key] = src
    n = kda.kda_selective_scan_bwd_workspace_size(B, T, D, S, G, 0 if cu is None else i["N"])
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    call = lambda grads: kda.kda_selective_scan_bwd(  # noqa: E731
        i["x"], i["delta"], i["A"], i["Bm"], i["Cm"], i["dout"], grads, ws, init_state=i["init"],
        d_final=i["d_final"], cu_seqlens=i["cu"], **scan_opt(i))
    call(g)
    ok(ws)
    o.check_guards()
    t, ro, rf = scan_ref(i, grad=True)
    loss = (ro * host(flat(i["dout"]))).sum()
    if i["d_final"] is not None:
        loss = loss + (rf * host(i["d_final"])).sum()
    loss.backward()
    for key, src in names.items():
        near(g[key].reshape(t[src].shape), t[src].grad, what=key)
    again = {k: torch.full_like(v, float("nan")) for k, v in g.items()}
    call(again)
    for k in g:
        assert torch.equal(g[k], again[k]), k  # fixed order of every sum


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,D,S,G,gate", [(1, 8, 16, 1, True), (3, 40, 8, 1, True),
                                          (5, 128, 32, 4, False), (2, 72, 64, 1, True),
                                          (3, 24, 128, 1, True), (40, 1032, 16, 1, True)])
def test_scan_steps_continue_a_prompt(N, D, S, G, gate, dtype):
    case = (N, 9, D, S, G, None, gate, True, True, True, True, True)
    i = scan_inputs(case, dtype, seed=5)
    o = Outs()
    state = o((N, D, S))
    ws = torch.empty(max(256, kda.kda_selective_scan_fwd_workspace_size(N, 9, D, S, G)),
                     dtype=torch.uint8, device=DEV)
    cut = lambda t: None if t is None else t[:, :4].contiguous()  # noqa: E731
    kda.kda_selective_scan_fwd(cut(i["x"]), cut(i["delta"]), i["A"], cut(i["Bm"]), cut(i["Cm"]),
                               torch.empty(N, 4, D, dtype=dtype, device=DEV), ws,
                               init_state=i["init"], final_state=state, D=i["D"],
                               z=cut(i["z"]), delta_bias=i["delta_bias"])
    _, ro, rf = scan_ref(i)
    ro = ro.view(N, 9, D)
    out = o((N, D), dtype)
    for t in range(4, 9):  # rows 9 tokens of a wider tensor apart
        kda.kda_selective_scan_step(i["x"][:, t], i["delta"][:, t], i["A"], i["Bm"][:, t],
                                    i["Cm"][:, t], state, out, D=i["D"],
                                    z=None if i["z"] is None else i["z"][:, t],
                                    delta_bias=i["delta_bias"])
        near(out, ro[:, t], dtype)
    near(state, rf)
    o.check_guards()


def test_scan_extreme_steps():
    """Steps from e^-30 to 200 through the softplus, decays that vanish, and a
    gate at both ends: finite, and on the reference."""
    D, T, S = 32, 40, 16
    gen = torch.Generator().manual_seed(11)
    case = (1, T, D, S, 1, None, True, True, True, True, True, False)
    i = scan_inputs(case, F32)
    i["delta"] = (torch.linspace(-30, 200, T * D)[torch.randperm(T * D, generator=gen)]
                  .view(1, T, D).to(DEV))
    i["z"] = torch.linspace(-120, 120, T * D).view(1, T, D).to(DEV)
    out, fin = (torch.empty(s, device=DEV) for s in ((1, T, D), (1, D, S)))
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    kda.kda_selective_scan_fwd(i["x"], i["delta"], i["A"], i["Bm"], i["Cm"], out, ws,
                               init_state=i["init"], final_state=fin, **scan_opt(i))
    _, ro, rf = scan_ref(i)
    near(flat(out), ro)
    near(fin, rf)


# ------------------------------------------------------------------- norms
NORM_CASES = [
    # lead, Hq, Hk, d, rot, pairs, l2, weights, wide, first position
    ((1,), 1, 1, 8, 0, False, True, False, False, 0),
    ((3,), 2, 1, 24, 16, False, False, True, False, 0),
    ((2, 5), 4, 2, 64, 64, False, False, True, True, 1000000),
    ((2, 5), 4, 4, 64, 32, True, True, True, True, 2000000000),
    ((1, 19), 7, 3, 128, 128, False, False, True, False, 131071),
    ((1, 19), 32, 8, 128, 128, True, False, False, False, 5),
    ((17,), 3, 3, 136, 96, False, True, True, False, 77),
    ((2, 3), 5, 1, 256, 256, False, False, True, True, 4096),
    ((2, 3), 5, 1, 200, 64, True, False, True, False, -500000),
    ((1, 301), 32, 32, 128, 0, False, True, False, True, 0),
    ((1, 2500), 2, 1, 32, 32, False, False, True, False, 99),
]


def norm_inputs(case, dtype, seed=1):
    lead, Hq, Hk, d, rot, pairs, l2, weights, wide, first = case
    gen = torch.Generator().manual_seed(seed)
    n = 1
    for m in lead:
        n *= m
    q = rows_of(draw(gen, *lead, Hq * d, dtype=dtype), wide, gen).unflatten(-1, (Hq, d))
    k = rows_of(draw(gen, *lead, Hk * d, scale=3.0, dtype=dtype), wide, gen)
    k = k.unflatten(-1, (Hk, d))
    qw, kw = (0.5 + torch.rand(2, d, generator=gen)).to(DEV) if weights else (None, None)
    pos = freq = None
    if rot:
        pos = (first + torch.arange(n)).to(torch.int32).view(lead).to(DEV)
        freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=R.F64) / rot)).float().to(DEV)
    opt = dict(q_weight=qw, k_weight=kw, positions=pos, inv_freq=freq,
               mode=kda.KDA_NORM_L2 if l2 else kda.KDA_NORM_RMS,
               rotation=kda.KDA_ROT_PAIRS if pairs else kda.KDA_ROT_HALVES, eps=1e-5)
    return q, k, opt, draw(gen, *lead, Hq, d), draw(gen, *lead, Hk, d)


def norm_ref(x, w, case, opt, grad=False):
    d = case[3]
    x64 = host(x.reshape(-1, x.shape[-2], d), grad)
    w64 = host(w, grad) if w is not None else None
    pos = None if opt["positions"] is None else opt["positions"].reshape(-1).cpu()
    freq = None if opt["inv_freq"] is None else opt["inv_freq"].cpu()
    return x64, w64, R.norm(x64, w64, pos, freq, case[6], case[5], opt["eps"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", NORM_CASES)
def test_norm_forward(case, dtype):
    q, k, opt, _, _ = norm_inputs(case, dtype)
    o = Outs()
    qo, ko = o(tuple(q.shape), dtype), o(tuple(k.shape), dtype)
    kda.kda_qk_norm_fwd(q, k, qo, ko, **opt)
    torch.cuda.synchronize()
    o.check_guards()
    for x, w, y in ((q, opt["q_weight"], qo), (k, opt["k_weight"], ko)):
        ref = norm_ref(x, w, case, opt)[2]
        near(y.reshape(ref.shape), ref, dtype)
    # in place
    qi, ki = q.contiguous().clone(), k.contiguous().clone()
    kda.kda_qk_norm_fwd(qi, ki, qi, ki, **opt)
    assert torch.equal(qi, qo) and torch.equal(ki, ko)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", NORM_CASES)
def test_norm_gradients(case, dtype):
    lead, Hq, Hk, d = case[:4]
    q, k, opt, dqo, dko = norm_inputs(case, dtype, seed=2)
    o = Outs()
    g = dict(dq=o(tuple(q.shape)), dk=o(tuple(k.shape)))
    ws = None
    if opt["q_weight"] is not None:
        g.update(dq_weight=o((d,)), dk_weight=o((d,)))
        n = 1
        for m in lead:
            n *= m
        ws = torch.full((kda.kda_qk_norm_bwd_workspace_size(n, Hq, Hk, d),), 255,
                        dtype=torch.uint8, device=DEV)
    kda.kda_qk_norm_bwd(q, k, dqo, dko, g, ws, **opt)
    torch.cuda.synchronize()
    o.check_guards()
    for x, name, dy in ((q, "q", dqo), (k, "k", dko)):
        x64, w64, y = norm_ref(x, opt[name + "_weight"], case, opt, grad=True)
        y.backward(host(dy).view(y.shape))
        near(g["d" + name].reshape(x64.shape), x64.grad, what=name)
        if w64 is not None:
            near(g[f"d{name}_weight"], w64.grad, what=name + " weight")
    # over the cotangents
    h = dict(dq=dqo, dk=dko)
    kda.kda_qk_norm_bwd(q, k, dqo, dko, h, None, **opt)
    assert torch.equal(h["dq"], g["dq"]) and torch.equal(h["dk"], g["dk"])


def test_norm_zero_rows():
    q = torch.zeros(3, 2, 64, dtype=BF16, device=DEV)
    out = torch.full_like(q, float("nan"))
    kda.kda_qk_norm_fwd(q, q.clone(), out, torch.empty_like(q))
    assert bool((out == 0).all())
    dy = torch.ones(3, 2, 64, device=DEV)
    g = dict(dq=torch.empty_like(dy), dk=torch.empty_like(dy))
    kda.kda_qk_norm_bwd(q, q, dy, dy, g, eps=1e-4)
    near(g["dq"], torch.full((3, 2, 64), 100.0))  # dy / sqrt(eps)


# --------------------------------------------- offsets, streams, graphs, status
@pytest.mark.parametrize("bad", [[1, 20, 40], [0, 30, 20, 40], [0, 20, 39], [0, 41, 40],
                                 [0, -5, 40]])
def test_malformed_offsets_write_nothing(bad):
    cu = cu_tensor(bad)
    N, T, D, S = len(bad) - 1, 40, 64, 16
    gen = torch.Generator().manual_seed(1)
    x = draw(gen, 1, T, D)
    w = draw(gen, D, 4)
    mark = lambda *s: torch.full(s, 5.0, device=DEV)  # noqa: E731

    def refused(ws, outs):
        st, _ = kda.kda_get_device_status(ws)
        assert st == kda.KDA_ERR_BAD_SEQLENS
        for t in outs:
            assert bool((t == 5).all())

    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    out, fin = mark(1, T, D), mark(N, 3, D)
    kda.kda_short_conv_fwd(x, w, out, ws, cu_seqlens=cu, final_state=fin)
    refused(ws, [out, fin])
    ws = torch.empty(kda.kda_short_conv_bwd_workspace_size(1, T, D, 4, N), dtype=torch.uint8,
                     device=DEV)
    g = dict(dx=mark(1, T, D), dweight=mark(D, 4), dbias=mark(D), d_init=mark(N, 3, D))
    kda.kda_short_conv_bwd(x, w, x, g, ws, cu_seqlens=cu)
    refused(ws, g.values())
    A, bc = -torch.ones(D, S, device=DEV), draw(gen, 1, T, 1, S)
    ws = torch.empty(kda.kda_selective_scan_fwd_workspace_size(1, T, D, S, 1, N),
                     dtype=torch.uint8, device=DEV)
    out, fin = mark(1, T, D), mark(N, D, S)
    kda.kda_selective_scan_fwd(x, x, A, bc, bc, out, ws, cu_seqlens=cu, final_state=fin)
    refused(ws, [out, fin])
    ws = torch.empty(kda.kda_selective_scan_bwd_workspace_size(1, T, D, S, 1, N),
                     dtype=torch.uint8, device=DEV)
    g = dict(dx=mark(1, T, D), ddelta=mark(1, T, D), dA=mark(D, S), dB=mark(1, T, 1, S),
             dC=mark(1, T, 1, S), dD=mark(D), ddelta_bias=mark(D), d_init=mark(N, D, S))
    kda.kda_selective_scan_bwd(x, x, A, bc, bc, x, g, ws, cu_seqlens=cu)
    refused(ws, g.values())


def test_capture_and_replay_on_another_stream():
    """One graph of the whole layer front, replayed on new inputs."""
    gen = torch.Generator().manual_seed(3)
    B, T, H, d = 2, 50, 2, 64
    D = H * d
    x = draw(gen, B, T, D, dtype=BF16)
    w = draw(gen, D, 4, scale=0.5)
    A = -torch.rand(D, 16, generator=gen).to(DEV)
    bc = draw(gen, B, T, 1, 16, dtype=BF16)
    ws = torch.empty(max(kda.kda_selective_scan_bwd_workspace_size(B, T, D, 16),
                         kda.kda_short_conv_bwd_workspace_size(B, T, D, 4)),
                     dtype=torch.uint8, device=DEV)
    e = lambda *s, dtype=F32: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
    c, y = e(B, T, D, dtype=BF16), e(B, T, D, dtype=BF16)
    qo, ko = e(B, T, H, d, dtype=BF16), e(B, T, H, d, dtype=BF16)
    g = dict(dx=e(B, T, D), ddelta=e(B, T, D), dA=e(D, 16), dB=e(B, T, 1, 16),
             dC=e(B, T, 1, 16))
    gc = dict(dx=e(B, T, D), dweight=e(D, 4))
    gn = dict(dq=e(B, T, H, d), dk=e(B, T, H, d))

    def run(stream=None):
        kda.kda_short_conv_fwd(x, w, c, ws, stream=stream)
        heads = c.view(B, T, H, d)
        kda.kda_qk_norm_fwd(heads, heads, qo, ko, stream=stream)
        kda.kda_selective_scan_fwd(c, x, A, bc, bc, y, ws, stream=stream)
        kda.kda_selective_scan_bwd(c, x, A, bc, bc, y, g, ws, stream=stream)
        kda.kda_qk_norm_bwd(heads, heads, g["dx"].view(B, T, H, d), g["dx"].view(B, T, H, d), gn,
                            stream=stream)
        kda.kda_short_conv_bwd(x, w, g["dx"], gc, ws, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(side)
    side.synchronize()
    outs = [c, y, qo, ko, *g.values(), *gc.values(), *gn.values()]
    first = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, first):
        assert torch.equal(a, b)
    x.copy_(draw(gen, B, T, D, dtype=BF16))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in outs]
    run()
    torch.cuda.synchronize()
    for a, b in zip(outs, replayed):
        assert torch.equal(a, b)


# ----------------------------------------------------------------- together
def test_layer_front_into_the_recurrence(oracle_mod):
    """Fused projection -> convolutions -> unit rows -> gated chunk prefill, and
    back: recurrence, norms and convolutions, against fp64 on the same inputs."""
    B, T, H, d = 1, 70, 2, 64
    D = H * d
    gen = torch.Generator().manual_seed(21)
    proj = draw(gen, B, T, 3 * D)  # q | k | v of every token
    wts = [draw(gen, D, 4, scale=0.5) for _ in range(3)]
    base = W.make_prefill_inputs(B, T, H, d, d, F32, seed=4, device=DEV)
    ws = torch.empty(max(kda.kda_chunk_fwd_workspace_size(B, T, H, d, d, in_dtype=kda.KDA_F32),
                         kda.kda_recurrent_bwd_workspace_size(B, T, H, d, d),
                         kda.kda_short_conv_bwd_workspace_size(B, T, D, 4)),
                     dtype=torch.uint8, device=DEV)
    c = [torch.empty(B, T, D, device=DEV) for _ in range(3)]
    for j in range(3):
        kda.kda_short_conv_fwd(proj[..., j * D:(j + 1) * D], wts[j], c[j], ws)
    heads = [t.view(B, T, H, d) for t in c]
    q, k = torch.empty_like(heads[0]), torch.empty_like(heads[1])
    kda.kda_qk_norm_fwd(heads[0], heads[1], q, k)
    out = torch.empty(B, T, H, d, device=DEV)
    kda.kda_chunk_fwd_gated(q, k, heads[2], base["z"], base["A_log"], base["beta"], out, ws)
    dout = draw(gen, B, T, H, d)
    g = torch.empty_like(base["z"])
    kda.kda_gate_fwd(base["z"], base["A_log"], g)
    e = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    gr = dict(dq=e(B, T, H, d), dk=e(B, T, H, d), dv=e(B, T, H, d), dg=e(B, T, H, d),
              dbeta=e(B, T, H))
    kda.kda_recurrent_bwd(q, k, heads[2], g, base["beta"], dout, gr, ws)
    kda.kda_qk_norm_bwd(heads[0], heads[1], gr["dq"], gr["dk"], dict(dq=gr["dq"], dk=gr["dk"]))
    grads = []
    for j, n in enumerate(("dq", "dk", "dv")):
        grads.append(dict(dx=e(B, T, D), dweight=e(D, 4)))
        kda.kda_short_conv_bwd(proj[..., j * D:(j + 1) * D], wts[j], gr[n].view(B, T, D),
                               grads[j], ws)

    p64 = host(proj[0], True)
    w64 = [host(w, True) for w in wts]
    cr = [R.conv(p64[:, j * D:(j + 1) * D], w64[j], None, None, [(0, T)], True)[0]
          for j in range(3)]
    q64, k64 = (R.norm(t.view(T, H, d), None, None, None, True, False, 1e-6) for t in cr[:2])
    v64 = cr[2].view(T, H, d)
    f = lambda t: host(t).numpy()  # noqa: E731
    n = lambda t: t.detach()[None].numpy()  # noqa: E731
    g64 = oracle_mod.gate(f(base["z"]), f(base["A_log"]), -5.0)
    o64, _ = oracle_mod.forward(n(q64), n(k64), n(v64), g64, f(base["beta"]))
    near(out, torch.from_numpy(o64))
    ref = oracle_mod.backward(n(q64), n(k64), n(v64), g64, f(base["beta"]), f(dout))
    torch.autograd.backward([q64, k64, v64], [torch.from_numpy(ref[m])[0]
                                              for m in ("dq", "dk", "dv")])
    # 2e-5: the recurrence's own bar and the two operators' in a row
    for j in range(3):
        assert R.rel_l2(grads[j]["dx"][0], p64.grad[:, j * D:(j + 1) * D]) <= 2e-5
        assert R.rel_l2(grads[j]["dweight"], w64[j].grad) <= 2e-5


def test_layer_decode_after_a_packed_prompt():
    """Convolution and scan over a packed prompt, then single tokens: the rows of
    one pass over the longer sequences."""
    lens, K, D, S = [5, 0, 33, 1], 3, 64, 16
    N, T = len(lens), sum(lens)
    gen = torch.Generator().manual_seed(8)
    seqs = [draw(gen, n + K, D) for n in lens]
    w = draw(gen, D, 4, scale=0.5)
    A = -(0.2 + torch.rand(D, S, generator=gen)).to(DEV)
    mix = draw(gen, D, 2 * S, scale=0.2)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x = torch.cat([s[:n] for s, n in zip(seqs, lens)])[None].contiguous()
    ws = torch.empty(kda.kda_selective_scan_fwd_workspace_size(1, T, D, S, 1, N),
                     dtype=torch.uint8, device=DEV)
    c, y = torch.empty_like(x), torch.empty_like(x)
    cs, hs = torch.empty(N, 3, D, device=DEV), torch.empty(N, D, S, device=DEV)
    kda.kda_short_conv_fwd(x, w, c, ws, cu_seqlens=cu_tensor(cu), final_state=cs)
    bc = (c @ mix).unflatten(-1, (2, S))
    kda.kda_selective_scan_fwd(c, c, A, bc[..., :1, :], bc[..., 1:, :], y, ws,
                               cu_seqlens=cu_tensor(cu), final_state=hs)
    got = [[y[0, a:b]] for a, b in zip(cu[:-1], cu[1:])]
    for t in range(K):
        xt = torch.stack([s[n + t] for s, n in zip(seqs, lens)])
        ct, yt = torch.empty_like(xt), torch.empty_like(xt)
        kda.kda_short_conv_step(xt, w, cs, ct)
        bc = (ct @ mix).unflatten(-1, (2, S))
        kda.kda_selective_scan_step(ct, ct, A, bc[:, :1], bc[:, 1:], hs, yt)
        for n in range(N):
            got[n].append(yt[n:n + 1])
    w64, A64, m64 = host(w), host(A), host(mix)
    for n, s in enumerate(seqs):
        b = [(0, len(s))]
        c64 = R.conv(host(s), w64, None, None, b, True)[0]
        bc = (c64 @ m64).unflatten(-1, (2, S))
        ref, _ = R.scan(c64, c64, A64, bc[:, :1], bc[:, 1:], None, None, None, True, None, b)
        # torch's fp32 product in between: 64 terms, some 1e-6
        assert R.rel_l2(torch.cat(got[n]), ref) <= 2e-5
