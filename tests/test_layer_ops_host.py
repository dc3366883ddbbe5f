"""Host side of the operators around the recurrence: the references'
gradients against differences, and every refusal of bad arguments before
anything is launched (fake pointers, no GPU)."""
import itertools

import pytest
import torch

import gated_delta_rule_158_b200 as kda
from gated_delta_rule_158_b200 import _lib

import layer_ref as R

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_158_b200 import build
    build.build()
    return _lib.lib()


def at(i):
    """A distinct fake buffer 4 GiB after the last."""
    return FAKE + (i << 32)


# ------------------------------------------------------- reference gradients
def _r(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, dtype=R.F64) * scale).requires_grad_()


@pytest.mark.parametrize("silu,state", list(itertools.product([False, True], repeat=2)))
def test_conv_reference_gradients_against_differences(silu, state):
    g = torch.Generator().manual_seed(3)
    x, w, b = _r(g, 7, 3), _r(g, 3, 4), _r(g, 3)
    s0 = _r(g, 3, 3, 3) if state else None
    bounds = [(0, 5), (5, 5), (5, 7)]
    f = lambda x, w, b, s0: R.conv(x, w, b, s0, bounds, silu)  # noqa: E731
    assert torch.autograd.gradcheck(f, (x, w, b, s0), eps=1e-6, atol=1e-7)


@pytest.mark.parametrize("gate,softplus", list(itertools.product([False, True], repeat=2)))
def test_scan_reference_gradients_against_differences(gate, softplus):
    g = torch.Generator().manual_seed(4)
    x, delta = _r(g, 6, 4), _r(g, 6, 4, scale=0.3)
    A = (-torch.rand(4, 3, generator=g, dtype=R.F64) - 0.2).requires_grad_()
    Bm, Cm, D = _r(g, 6, 2, 3), _r(g, 6, 2, 3), _r(g, 4)
    z = _r(g, 6, 4) if gate else None
    bias, h0 = _r(g, 4), _r(g, 2, 4, 3)
    f = lambda *a: R.scan(*a[:6], z, a[6], softplus, a[7], [(0, 4), (4, 6)])  # noqa: E731
    assert torch.autograd.gradcheck(f, (x, delta, A, Bm, Cm, D, bias, h0), eps=1e-6, atol=1e-7)


@pytest.mark.parametrize("l2,pairs", list(itertools.product([False, True], repeat=2)))
def test_norm_reference_gradients_against_differences(l2, pairs):
    g = torch.Generator().manual_seed(5)
    x, w = _r(g, 3, 2, 8), _r(g, 8)
    pos = torch.tensor([0, 5, 1000003], dtype=torch.int32)
    f = lambda x, w: R.norm(x, w, pos, torch.tensor([1.0, 0.5]), l2, pairs, 1e-6)  # noqa: E731
    assert torch.autograd.gradcheck(f, (x, w), eps=1e-6, atol=1e-7)


# ----------------------------------------------------------------- refusals
INV, UNS, MIS, WS = (_lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED,
                     _lib.KDA_ERR_MISALIGNED, _lib.KDA_ERR_WORKSPACE)


def _call(fn, base, over):
    a = dict(base)
    a.update(over)
    return fn(*a.values())


CONV = dict(x=at(0), xs=64, w=at(1), b=at(2), dt=1, init=at(3), cu=None, num=0, B=2, T=100, D=64,
            W=4, act=1, out=at(4), fin=at(5), ws=at(6), wsb=1 << 30, st=None)
SHARED_CONV = [
    (dict(x=None), INV), (dict(w=None), INV), (dict(dt=2), INV), (dict(act=2), INV),
    (dict(B=0), INV), (dict(T=0), INV), (dict(D=0), INV), (dict(W=0), INV),
    (dict(D=60, xs=64), UNS), (dict(W=1), UNS), (dict(W=5), UNS),
    (dict(xs=56), INV), (dict(xs=65), INV), (dict(xs=1 << 33), INV),
    (dict(x=at(0) + 8), MIS), (dict(w=at(1) + 4), MIS), (dict(b=at(2) + 4), MIS),
    (dict(cu=at(9), num=3), INV), (dict(cu=at(9), num=0, B=1), INV), (dict(num=3), INV),
    (dict(B=1 << 16, T=1 << 16), UNS), (dict(wsb=255), WS), (dict(ws=None), INV),
]


@pytest.mark.parametrize("over,code", SHARED_CONV + [
    (dict(out=None), INV), (dict(out=at(4) + 2), MIS), (dict(fin=at(5) + 4), MIS),
    (dict(out=at(0)), INV), (dict(out=at(0) + 64), INV),     # inside x
    (dict(fin=at(3)), INV), (dict(fin=at(4) + 128), INV), (dict(ws=at(4)), INV),
])
def test_short_conv_fwd_rejects_on_host(L, over, code):
    assert _call(L.kda_short_conv_fwd, CONV, over) == code


CSTEP = dict(x=at(0), xs=64, w=at(1), b=at(2), dt=1, state=at(3), N=5, D=64, W=4, act=1,
             out=at(4), st=None)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), INV), (dict(state=None), INV), (dict(out=None), INV), (dict(N=0), INV),
    (dict(D=12, xs=16), UNS), (dict(W=6), UNS), (dict(dt=3), INV), (dict(xs=60), INV),
    (dict(state=at(0)), INV), (dict(out=at(3)), INV), (dict(out=at(4) + 4), MIS),
])
def test_short_conv_step_rejects_on_host(L, over, code):
    assert _call(L.kda_short_conv_step, CSTEP, over) == code


CBWD = dict(x=at(0), xs=64, w=at(1), b=at(2), dt=1, init=at(3), dout=at(4), dfin=at(5), cu=None,
            num=0, B=2, T=100, D=64, W=4, act=1, dx=at(6), dw=at(7), db=at(8), dinit=at(10),
            ws=at(11), wsb=1 << 30, st=None)


@pytest.mark.parametrize("over,code", SHARED_CONV + [
    (dict(dout=None), INV), (dict(dx=None), INV), (dict(dw=None), INV),
    (dict(dx=at(4)), INV),                    # dx may not overwrite dout
    (dict(db=at(7)), INV), (dict(dinit=at(5)), INV), (dict(dx=at(6) + 8), MIS),
])
def test_short_conv_bwd_rejects_on_host(L, over, code):
    assert _call(L.kda_short_conv_bwd, CBWD, over) == code


def test_short_conv_bwd_workspace(L):
    n = kda.kda_short_conv_bwd_workspace_size(2, 100, 64, 4)
    assert n > 256 and _call(L.kda_short_conv_bwd, CBWD, dict(wsb=n - 1)) == WS
    assert kda.kda_short_conv_bwd_workspace_size(2, 100, 60, 4) == 0
    assert kda.kda_short_conv_bwd_workspace_size(0, 100, 64, 4) == 0


SCAN = dict(x=at(0), xs=64, dl=at(1), dls=64, A=at(2), Bm=at(3), bs=16, Cm=at(4), cs=16,
            Ds=at(5), z=at(6), zs=64, db=at(7), sp=1, dt=1, init=at(8), cu=None, num=0, B=2,
            T=100, D=64, S=16, G=1, out=at(9), fin=at(10), ws=at(11), wsb=1 << 40, st=None)
SHARED_SCAN = [
    (dict(x=None), INV), (dict(dl=None), INV), (dict(A=None), INV), (dict(Bm=None), INV),
    (dict(Cm=None), INV), (dict(dt=5), INV), (dict(D=0), INV), (dict(G=0), INV),
    (dict(S=24, bs=24, cs=24), UNS), (dict(S=256, bs=256, cs=256), UNS), (dict(S=4), UNS),
    (dict(D=52), UNS), (dict(G=3, bs=48, cs=48), UNS), (dict(G=16, bs=256, cs=256), UNS),
    (dict(xs=48), INV), (dict(dls=68), INV), (dict(bs=8), INV), (dict(cs=20), INV),
    (dict(zs=0), INV), (dict(z=at(6) + 2), MIS), (dict(A=at(2) + 4), MIS),
]
SHARED_SEQ = [
    (dict(B=0), INV), (dict(T=-1), INV), (dict(cu=at(12), num=2), INV), (dict(num=1), INV),
    (dict(B=1 << 16, T=1 << 16), UNS), (dict(ws=None), INV), (dict(wsb=0), WS),
]


@pytest.mark.parametrize("over,code", SHARED_SCAN + SHARED_SEQ + [
    (dict(out=None), INV), (dict(out=at(6)), INV), (dict(fin=at(9)), INV),
    (dict(fin=at(8) + 4096), INV),            # overlaps init_state without being it
    (dict(init=at(11)), INV), (dict(init=at(8) + 4), MIS),
])
def test_selective_scan_fwd_rejects_on_host(L, over, code):
    assert _call(L.kda_selective_scan_fwd, SCAN, over) == code


SSTEP = {k: SCAN[k] for k in ("x xs dl dls A Bm bs Cm cs Ds z zs db sp dt".split())}
SSTEP.update(state=at(8), N=3, D=64, S=16, G=1, out=at(9), st=None)


@pytest.mark.parametrize("over,code", SHARED_SCAN + [
    (dict(N=0), INV), (dict(state=None), INV), (dict(out=None), INV), (dict(state=at(2)), INV),
    (dict(out=at(0)), INV), (dict(out=at(9) + 8), MIS),
])
def test_selective_scan_step_rejects_on_host(L, over, code):
    assert _call(L.kda_selective_scan_step, SSTEP, over) == code


SBWD = {k: SCAN[k] for k in ("x xs dl dls A Bm bs Cm cs Ds z zs db sp dt init".split())}
SBWD.update(dout=at(13), dfin=at(14), cu=None, num=0, B=2, T=100, D=64, S=16, G=1, dx=at(15),
            ddl=at(16), dA=at(17), dB=at(18), dC=at(19), dD=at(20), dz=at(21), ddb=at(22),
            dinit=at(23), ws=at(24), wsb=1 << 40, st=None)


@pytest.mark.parametrize("over,code", SHARED_SCAN + SHARED_SEQ + [
    (dict(dout=None), INV), (dict(dx=None), INV), (dict(dB=None), INV), (dict(dz=None), INV),
    (dict(z=None), INV),                      # dz without z
    (dict(dx=at(13)), INV), (dict(dB=at(19)), INV), (dict(dinit=at(14)), INV),
    (dict(dA=at(17) + 4), MIS),
])
def test_selective_scan_bwd_rejects_on_host(L, over, code):
    assert _call(L.kda_selective_scan_bwd, SBWD, over) == code


def test_selective_scan_workspaces(L):
    for fn, entry, base in ((kda.kda_selective_scan_fwd_workspace_size,
                             L.kda_selective_scan_fwd, SCAN),
                            (kda.kda_selective_scan_bwd_workspace_size,
                             L.kda_selective_scan_bwd, SBWD)):
        n = fn(2, 100, 64, 16, 1)
        assert n >= 256 and _call(entry, base, dict(wsb=n - 1)) == WS
        assert fn(1, 5000, 64, 16, 1, 7) > 256       # packed: the segments' offsets
        assert fn(1, 65536, 64, 16, 1) > 256         # one long sequence: its segments' states
        assert fn(2, 100, 64, 24, 1) == 0 and fn(2, 100, 64, 16, 0) == 0 and fn(0, 1, 64, 16) == 0


NORM = dict(q=at(0), qs=256, k=at(1), ks=128, qw=at(2), kw=at(3), pos=at(4), freq=at(5), dt=1,
            tokens=10, Hq=4, Hk=2, d=64, rot=32, norm=0, rotation=0, eps=1e-6, qo=at(6),
            ko=at(7), st=None)
SHARED_NORM = [
    (dict(q=None), INV), (dict(k=None), INV), (dict(tokens=0), INV), (dict(Hq=0), INV),
    (dict(Hk=0), INV), (dict(d=0), INV), (dict(dt=9), INV), (dict(norm=2), INV),
    (dict(rotation=2), INV), (dict(eps=0.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(rot=-16), INV), (dict(rot=80), INV),
    (dict(rot=24), UNS), (dict(d=60), UNS), (dict(d=264, qs=4096, ks=4096), UNS),
    (dict(pos=None), INV), (dict(freq=None), INV), (dict(rot=0), INV),
    (dict(qs=248), INV), (dict(ks=132), INV), (dict(q=at(0) + 8), MIS), (dict(pos=at(4) + 4), MIS),
]


@pytest.mark.parametrize("over,code", SHARED_NORM + [
    (dict(qo=None), INV), (dict(ko=None), INV), (dict(qo=at(1)), INV), (dict(ko=at(0)), INV),
    (dict(qo=at(0) + 512), INV),              # shifted, so not in place
    (dict(qs=512, qo=at(0)), INV),            # strided rows cannot be their own dense output
    (dict(ko=at(6)), INV), (dict(qo=at(6) + 8), MIS),
])
def test_qk_norm_fwd_rejects_on_host(L, over, code):
    assert _call(L.kda_qk_norm_fwd, NORM, over) == code


NBWD = {k: NORM[k] for k in NORM if k not in ("qo", "ko", "st")}
NBWD.update(dqo=at(8), dko=at(9), dq=at(10), dk=at(11), dqw=at(12), dkw=at(13), ws=at(14),
            wsb=1 << 30, st=None)


@pytest.mark.parametrize("over,code", SHARED_NORM + [
    (dict(dqo=None), INV), (dict(dk=None), INV), (dict(qw=None), INV), (dict(kw=None), INV),
    (dict(dq=at(9)), INV), (dict(dk=at(10)), INV), (dict(dq=at(8) + 64), INV),
    (dict(ws=None), WS), (dict(wsb=16), WS), (dict(ws=at(8)), INV), (dict(dkw=at(12)), INV),
])
def test_qk_norm_bwd_rejects_on_host(L, over, code):
    assert _call(L.kda_qk_norm_bwd, NBWD, over) == code


# --------------------------------------------- the binding's own checks (CPU)
def test_binding_refuses_host_tensors_types_and_shapes(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = torch.zeros(2, 5, 64)
    w = torch.zeros(64, 4)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kda_short_conv_fwd(x, w, torch.zeros_like(x), ws)
    with pytest.raises(TypeError, match="dtype"):
        kda.kda_short_conv_step(x[:, 0].half(), w, torch.zeros(2, 3, 64), x[:, 1])
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kda_qk_norm_fwd(x[..., None, :], x[..., None, :], x, x)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kda_selective_scan_step(x[:, 0], x[:, 0], torch.zeros(64, 16), torch.zeros(2, 1, 16),
                                    torch.zeros(2, 1, 16), torch.zeros(2, 64, 16), x[:, 1])


def test_row_strides_of_slices():
    wide = torch.zeros(3, 5, 96)
    f, host = torch.float32, wide.get_device()

    def rows(t, lead, width, shape=None):
        return _lib._rows(host, "x", t, t.shape if shape is None else shape, lead, width, f)

    p, st = rows(wide[..., 32:64], 2, 32)
    assert st == 96 and p == wide.data_ptr() + 32 * 4
    assert rows(wide[:1, :1], 2, 96)[1] == 96  # no second row
    assert rows(wide[:1, :1, :32], 2, 32)[1] == 32
    assert rows(wide[:, 2:3], 2, 96)[1] == 480
    assert rows(wide.view(3, 5, 4, 24)[:, :, 1:3], 2, 48)[1] == 96
    with pytest.raises(ValueError, match="constant distance"):
        rows(wide[:, :4], 2, 96)
    with pytest.raises(ValueError, match="dense"):
        rows(wide[..., ::2], 2, 48)
    with pytest.raises(ValueError, match="dense"):
        rows(wide.view(3, 5, 4, 24)[:, :, ::2], 2, 48)
    with pytest.raises(ValueError, match="overlap"):
        rows(wide[:1, :1].expand(3, 5, 96), 2, 96)
    with pytest.raises(ValueError, match="shape"):
        rows(wide, 2, 96, shape=(3, 5, 95))
    with pytest.raises(TypeError, match="Tensor"):
        _lib._rows(host, "x", None, (3, 5, 96), 2, 96, f)
    with pytest.raises(TypeError, match="Tensor"):
        _lib._arg(host, "x", [1.0], (1,), f)
    with pytest.raises(ValueError, match="dense"):
        _lib._arg(host, "x", wide[..., ::2], (3, 5, 48), f)
