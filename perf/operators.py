"""Cases and plain forms of the operators around the recurrence: the short
causal convolution, the selective state space scan, and the per-head norms of
queries and keys with the position rotation.

`own` false: the operators in elementary torch operations, fp32 (angles in
fp64), rounded once at the end.  `own` true: the package's entry points.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the three convolved projections (q, k, v of 32 heads of 128) of one token
        # for each of 256 sequences being decoded
        dict(name="conv step 256", op="conv", mode="step", seqs=256, channels=12288, width=4,
             dtype="bf16", silu=True, bias=False),
        # a packed batch of prompts that continue from kept rows, one projection of 32 heads
        dict(name="conv prompt packed", op="conv", mode="prompt", packed=True, seqs=64,
             tokens=65000, channels=4096, width=4, dtype="bf16", silu=True, bias=True, state=True),
        # one training step's convolution of one projection, forward and gradients
        dict(name="conv train", op="conv", mode="train", packed=False, seqs=4, tokens=4096,
             channels=4096, width=4, dtype="bf16", silu=True, bias=True, state=False),
        # one decode step of one sequence: latency only
        dict(name="scan step 1", op="scan", mode="step", seqs=1, channels=2048, dstate=16,
             groups=1, dtype="bf16", gate=True),
        # one decode step of 256 sequences: the fp32 states cross HBM once each way
        dict(name="scan step 256", op="scan", mode="step", seqs=256, channels=4096, dstate=16,
             groups=1, dtype="bf16", gate=True),
        # one long prompt: little to run side by side but channels, states and segments
        dict(name="scan prompt long", op="scan", mode="prompt", packed=False, seqs=1,
             tokens=32768, channels=2048, dstate=16, groups=1, dtype="bf16", gate=True,
             state=False),
        # a packed batch of prompts of mixed lengths that continue from kept states
        dict(name="scan prompt packed", op="scan", mode="prompt", packed=True, seqs=16,
             tokens=12001, channels=4096, dstate=16, groups=1, dtype="bf16", gate=True,
             state=True),
        # fp32 with a wide state and two groups of B and C, odd length
        dict(name="scan prompt fp32 wide", op="scan", mode="prompt", packed=False, seqs=2,
             tokens=1001, channels=512, dstate=64, groups=2, dtype="f32", gate=False, state=True),
        # one training step's scan, forward and all gradients
        dict(name="scan train", op="scan", mode="train", packed=False, seqs=4, tokens=4096,
             channels=2048, dstate=16, groups=1, dtype="bf16", gate=True, state=False),
        # queries and keys of a decode batch: shared key heads, far positions, latency only
        dict(name="norm decode 16", op="norm", mode="prompt", tokens=16, q_heads=32, k_heads=8,
             dim=128, rot=128, pairs=False, kind="rms", weights=True, far=True, dtype="bf16"),
        # queries and keys of 16 K prompt tokens before the recurrence: unit rows, no rotation
        dict(name="norm prompt unit", op="norm", mode="prompt", tokens=16384, q_heads=32,
             k_heads=32, dim=128, rot=0, pairs=False, kind="l2", weights=False, far=False,
             dtype="bf16"),
        # one training step's norms and rotation of half of each row, forward and gradients
        dict(name="norm train", op="norm", mode="train", tokens=8192, q_heads=32, k_heads=8,
             dim=128, rot=64, pairs=False, kind="rms", weights=True, far=False, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "norm"])
    mode = rng.choice(["prompt", "step", "train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        dim = 8 * rng.randint(4, 32)
        qh = rng.randint(1, 48)
        kh = rng.randint(1, qh)
        room = 8192 * 40 * 128 // ((qh + kh) * dim)
        return dict(op=op, mode="train" if mode == "train" else "prompt",
                    tokens=min(16384, _log_int(rng, 1, room)), q_heads=qh, k_heads=kh,
                    dim=dim, rot=rng.choice([0, 16 * rng.randint(1, dim // 16)]),
                    pairs=rng.random() < 0.5, kind=rng.choice(["rms", "l2"]),
                    weights=rng.random() < 0.6, far=rng.random() < 0.5, dtype=dtype)
    channels = 8 * _log_int(rng, 8, 512)
    c = dict(op=op, mode=mode, channels=channels, dtype=dtype)
    if op == "conv":
        c.update(width=rng.randint(2, 4), silu=rng.random() < 0.7, bias=rng.random() < 0.5)
    else:
        groups = rng.choice([1, 1, 2, 4])
        if groups > 1:
            c["channels"] = channels = 64 * groups * rng.randint(1, 8)
        c.update(dstate=rng.choice([8, 16, 16, 32, 64, 128]), groups=groups,
                 gate=rng.random() < 0.7)
    if mode == "step":
        c["seqs"] = _log_int(rng, 1, 256 * 16 // max(16, c.get("dstate", 16)))
        return c
    room = (3 << 24) // channels if op == "conv" else (1 << 27) // (channels * c["dstate"])
    tokens = min(_log_int(rng, 1, max(2, room)), 16384)
    packed = rng.random() < 0.5
    seqs = min(_log_int(rng, 1, 40), tokens)
    c.update(packed=packed, seqs=seqs, tokens=tokens if packed else max(1, tokens // seqs),
             state=rng.random() < 0.6)
    return c


def _lengths(case, seed):
    """Sequence lengths: equal ones of a dense batch; ragged ones of a packed batch,
    an empty sequence and a one-token sequence among eight or more."""
    n, t = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [t] * n
    rng = random.Random(int(seed) * 7919 + n)
    share = [math.exp(rng.uniform(0.0, 3.5)) for _ in range(n)]
    if n >= 8:
        share[1] = 0.0
    total = sum(share)
    cuts, acc = [0], 0.0
    for s in share[:-1]:
        acc += s
        cuts.append(int(t * acc / total))
    cuts.append(t)
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _cu(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, device=dev) * (hi - lo) + lo

    s = {"case": dict(case)}
    if case["op"] == "norm":
        t, d = case["tokens"], case["dim"]
        s["q"] = normal(1, t, case["q_heads"], d, dtype=dt)
        s["k"] = normal(1, t, case["k_heads"], d, dtype=dt)
        s["q_weight"] = uniform(d, lo=0.5, hi=1.5) if case["weights"] else None
        s["k_weight"] = uniform(d, lo=0.5, hi=1.5) if case["weights"] else None
        s["positions"] = s["inv_freq"] = None
        if case["rot"]:
            i = torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64)
            s["inv_freq"] = (10000.0 ** (-i / case["rot"])).float()
            first = 1000000 if case["far"] else 0
            first += int(random.Random(int(seed)).random() * 1000)
            s["positions"] = (torch.arange(t, device=dev) + first).to(torch.int32).view(1, t)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        if case["mode"] == "train":
            s["dq_out"], s["dk_out"] = normal(*s["q"].shape), normal(*s["k"].shape)
            s["dq"], s["dk"] = torch.empty_like(s["dq_out"]), torch.empty_like(s["dk_out"])
            if case["weights"]:
                s["dq_weight"], s["dk_weight"] = uniform(d), uniform(d)
        return s

    D, n = case["channels"], case["seqs"]
    if case["mode"] == "step":
        lead, s["cu"] = (n,), None
    else:
        lens = _lengths(case, seed)
        lead = (1, case["tokens"]) if case["packed"] else (n, case["tokens"])
        s["cu"] = torch.tensor(_cu(lens), dtype=torch.int32, device=dev)  # flattened tokens
    s["x"] = normal(*lead, D, dtype=dt)
    s["out"] = torch.empty_like(s["x"])
    train = case["mode"] == "train"
    if case["op"] == "conv":
        W = case["width"]
        s["weight"] = normal(D, W, std=W ** -0.5)
        s["bias"] = normal(D, std=0.1) if case["bias"] else None
        s["state"] = None
        if case["mode"] == "step" or case["state"]:
            s["state"] = normal(n, W - 1, D, dtype=dt)
            s["final"] = torch.empty_like(s["state"])
        if train:
            s["dout"] = normal(*lead, D)
            s["dx"] = torch.empty_like(s["dout"])
            s["dweight"] = torch.empty_like(s["weight"])
            s["dbias"] = torch.empty_like(s["bias"]) if case["bias"] else None
            if case["state"]:
                s["d_final"] = normal(n, W - 1, D)
                s["d_init"] = torch.empty_like(s["d_final"])
        return s

    N, G = case["dstate"], case["groups"]
    # step sizes as a trained layer has them: softplus(bias) log-uniform in [0.001, 0.1]
    step = torch.exp(uniform(D, lo=math.log(0.001), hi=math.log(0.1)))
    s["delta_bias"] = step + torch.log(-torch.expm1(-step))
    s["delta"] = normal(*lead, D, std=0.7, dtype=dt)
    s["A"] = -torch.arange(1, N + 1, device=dev).float() * uniform(D, N, lo=0.7, hi=1.3)
    s["B"] = normal(*lead, G, N, dtype=dt)
    s["C"] = normal(*lead, G, N, dtype=dt)
    s["D"] = uniform(D, lo=0.5, hi=1.5)
    s["z"] = normal(*lead, D, dtype=dt) if case["gate"] else None
    s["state"] = None
    if case["mode"] == "step" or case["state"]:
        s["state"] = normal(n, D, N, std=0.5)
        s["final"] = torch.empty_like(s["state"])
    if train:
        s["dout"] = normal(*lead, D, dtype=dt)
        f32 = lambda t: torch.empty(t.shape, device=dev)  # noqa: E731
        s["dx"], s["ddelta"], s["dB"], s["dC"] = f32(s["x"]), f32(s["x"]), f32(s["B"]), f32(s["C"])
        s["dA"], s["dD"], s["ddelta_bias"] = f32(s["A"]), f32(s["D"]), f32(s["D"])
        s["dz"] = f32(s["z"]) if case["gate"] else None
        if case["state"]:
            s["d_final"] = normal(n, D, N, std=0.5)
            s["d_init"] = torch.empty_like(s["d_final"])
    return s


# -------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["mode"] == "train"
    if case["op"] == "norm":
        rows = case["tokens"] * (case["q_heads"] + case["k_heads"])
        n = rows * case["dim"]
        # x and y once; in training the two fp32 gradients too
        return {"bytes": n * (2 * e + (8 if train else 0)) + 4 * case["tokens"],
                "flops": n * (16 if train else 6)}
    D, n = case["channels"], case["seqs"]
    if case["mode"] == "step":
        t = n
    else:
        t = case["tokens"] if case["packed"] else n * case["tokens"]
    state = case["mode"] == "step" or case["state"]
    if case["op"] == "conv":
        W = case["width"]
        b = 2 * t * D * e + 4 * D * W
        b += 2 * n * (W - 1) * D * e if state else 0
        if train:
            b += 8 * t * D + 4 * D * W + (8 * n * (W - 1) * D if state else 0)
        return {"bytes": b, "flops": 2 * t * D * W * (3 if train else 1)}
    N, G = case["dstate"], case["groups"]
    b = t * D * e * (4 if case["gate"] else 3) + 2 * t * G * N * e + 4 * D * N
    b += 8 * n * D * N if state else 0
    if train:  # dout; dx, ddelta, dz; dB, dC; dA
        b += t * D * (e + (12 if case["gate"] else 8)) + 8 * t * G * N + 4 * D * N
        b += 8 * n * D * N if state else 0
    # per state element and token: decay (product, exponential), input, update, output; the
    # gradients take the forward's states again and about thrice its products
    return {"bytes": b, "flops": t * D * N * (28 if train else 7)}


# -------------------------------------------------------------- plain forms
def _flat(t):
    """[B, T, ...] as [B*T, ...]."""
    return None if t is None else t.reshape(-1, *t.shape[2:])


def _places(cu, total):
    """Of each token: its sequence and its place in it."""
    t = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(cu.dtype), right=True)
    return seq, t - cu[seq].long()


def _conv_rows(s, W):
    """[init rows; x rows] in fp32 and, for each token and tap, the row it reads."""
    x = _flat(s["x"]).float()
    T, D = x.shape
    cu = s["cu"].long()
    n = cu.numel() - 1
    init = s["state"].float().reshape(-1, D) if s["state"] is not None \
        else x.new_zeros(n * (W - 1), D)
    seq, off = _places(s["cu"], T)
    src = off[:, None] - (W - 1) + torch.arange(W, device=x.device)
    row = torch.where(src >= 0, n * (W - 1) + cu[seq][:, None] + src,
                      seq[:, None] * (W - 1) + src + W - 1)
    return torch.cat([init, x]), row, seq, off, cu


def _act(p, silu):
    return p * torch.sigmoid(p) if silu else p


def _conv_forward(s, rows, row, cu, W):
    c = s["case"]
    p = (rows[row] * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        p = p + s["bias"]
    out = {"out": _act(p, c["silu"]).to(s["x"].dtype).view_as(s["x"])}
    if s["state"] is not None:
        n = cu.numel() - 1
        src = (cu[1:] - cu[:-1])[:, None] - (W - 1) + torch.arange(W - 1, device=cu.device)
        at = torch.where(src >= 0, n * (W - 1) + cu[:-1, None] + src,
                         torch.arange(n, device=cu.device)[:, None] * (W - 1) + src + W - 1)
        out["final"] = rows[at].to(s["x"].dtype)
    return p, out


def _conv_plain(s):
    c = s["case"]
    W, D = c["width"], c["channels"]
    if c["mode"] == "step":
        rows = torch.cat([s["state"], s["x"][:, None]], 1)
        p = (rows.float() * s["weight"].t()).sum(1)
        if s["bias"] is not None:
            p = p + s["bias"]
        s["state"].copy_(rows[:, 1:])
        return {"out": _act(p, c["silu"]).to(s["x"].dtype), "state": s["state"]}
    rows, row, seq, off, cu = _conv_rows(s, W)
    p, out = _conv_forward(s, rows, row, cu, W)
    if c["mode"] == "prompt":
        return out
    ds = _flat(s["dout"])
    if c["silu"]:
        sg = torch.sigmoid(p)
        ds = ds * (sg * (1 + p * (1 - sg)))
    T = ds.shape[0]
    n = cu.numel() - 1
    lens = cu[1:] - cu[:-1]
    tap = torch.arange(W, device=ds.device)
    # a row at place i of its sequence (kept rows at -(W-1)..-1) is tap j of place i + W-1 - j
    to = off[:, None] + (W - 1) - tap
    keep = to < lens[seq][:, None]
    at = (cu[seq][:, None] + to).clamp(0, T - 1)
    w = s["weight"].t()
    dx = (torch.where(keep[..., None], ds[at], 0.0) * w).sum(1)
    if s["state"] is not None:
        i = torch.arange(W - 1, device=ds.device)
        fin = off - lens[seq] + (W - 1)  # its row of the final state, where not negative
        dx = dx + torch.where((fin >= 0)[:, None],
                              s["d_final"][seq, fin.clamp(0)], 0.0)
        to = (i[:, None] - tap).expand(n, W - 1, W)
        keep = (to >= 0) & (to < lens[:, None, None])
        at = (cu[:-1, None, None] + to).clamp(0, T - 1)
        d0 = (torch.where(keep[..., None], ds[at], 0.0) * w).sum(2)
        fin = i - lens[:, None]  # a kept row may still be kept at the end
        d0 = d0 + torch.where((fin >= 0)[..., None], torch.gather(
            s["d_final"], 1, fin.clamp(0)[..., None].expand(n, W - 1, D)), 0.0)
        out["d_init"] = d0
    out["dx"] = dx.view_as(s["x"])
    out["dweight"] = (rows[row] * ds[:, None]).sum(0).t().contiguous()
    if s["bias"] is not None:
        out["dbias"] = ds.sum(0)
    return out


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 0, h_{-1} = 0, by pairing neighbours."""
    T = a.shape[0]
    if T == 1:
        return b
    n = T // 2
    odd = _linear_scan(a[0:2 * n:2] * a[1:2 * n:2], a[1:2 * n:2] * b[0:2 * n:2] + b[1:2 * n:2])
    h = torch.empty_like(b)
    h[1:2 * n:2] = odd
    h[0] = b[0]
    h[2::2] = a[2::2] * odd[:(T - 1) // 2] + b[2::2]
    return h


def _scan_plain(s):
    c = s["case"]
    D, N, G = c["channels"], c["dstate"], c["groups"]
    step = c["mode"] == "step"
    f = (lambda t: None if t is None else t.float()) if step else \
        (lambda t: None if t is None else _flat(t).float())
    x, z = f(s["x"]), f(s["z"])
    dt = torch.nn.functional.softplus(f(s["delta"]) + s["delta_bias"])
    Bg, Cg = f(s["B"]), f(s["C"])
    T = x.shape[0]

    def heads(t):  # [T, G, N] -> [T, D, N]
        return t[:, :, None, :].expand(T, G, D // G, N).reshape(T, D, N)

    a = torch.exp(dt[..., None] * s["A"])
    b = (dt * x)[..., None] * heads(Bg)
    if step:
        h = a * s["state"] + b
        s["state"].copy_(h)
    else:
        cu = s["cu"].long()
        lens = cu[1:] - cu[:-1]
        seq, off = _places(s["cu"], T)
        first = (off == 0)
        if s["state"] is not None:
            b = b + torch.where(first[:, None, None], a, 0.0) * s["state"][seq]
        h = _linear_scan(torch.where(first[:, None, None], 0.0, a), b)
    y = (h * heads(Cg)).sum(-1)
    y = y + s["D"] * x
    gated = y if z is None else y * (z * torch.sigmoid(z))
    out = {"out": gated.to(s["x"].dtype).view_as(s["x"])}
    if step:
        out["state"] = s["state"]
        return out
    if s["state"] is not None:
        last = (cu[1:] - 1).clamp(0)
        out["final"] = torch.where((lens > 0)[:, None, None], h[last], s["state"])
    if c["mode"] == "prompt":
        return out

    dy = _flat(s["dout"]).float()
    if z is not None:
        sg = torch.sigmoid(z)
        out["dz"] = (dy * y * (sg * (1 + z * (1 - sg)))).view_as(s["x"])
        dy = dy * (z * sg)
    out["dD"] = (dy * x).sum(0)
    end = off == lens[seq] - 1
    src = dy[..., None] * heads(Cg)
    if s["state"] is not None:
        src = src + torch.where(end[:, None, None], s["d_final"][seq], 0.0)
    nxt = torch.cat([a[1:], a[:1]])
    nxt = torch.where(end[:, None, None], 0.0, nxt)
    g = _linear_scan(nxt.flip(0), src.flip(0)).flip(0)  # dL/dh_t
    del nxt, src
    out["dC"] = (h * dy[..., None]).view(T, G, D // G, N).sum(2).view_as(s["C"])
    out["dB"] = (g * (dt * x)[..., None]).view(T, G, D // G, N).sum(2).view_as(s["B"])
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    if s["state"] is not None:
        before = torch.where(first[:, None, None], s["state"][seq], before)
        start = cu[:-1].clamp(0, T - 1)
        out["d_init"] = torch.where((lens > 0)[:, None, None], g[start] * a[start], s["d_final"])
    else:
        before = torch.where(first[:, None, None], 0.0, before)
    gB = (g * heads(Bg)).sum(-1)
    ga = g * a * before  # dL/d(dt A)
    out["dA"] = (ga * dt[..., None]).sum(0)
    ddt = (ga * s["A"]).sum(-1) + gB * x
    out["dx"] = (gB * dt + dy * s["D"]).view_as(s["x"])
    ddelta = ddt * (-torch.expm1(-dt))  # softplus'(v) = 1 - exp(-softplus(v))
    out["ddelta"] = ddelta.view_as(s["x"])
    out["ddelta_bias"] = ddelta.sum(0)
    return out


def _rotate(v, s, back):
    c = s["case"]
    rot = c["rot"]
    if not rot:
        return v
    ang = s["positions"].double()[..., None, None] * s["inv_freq"].double()
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    sin = -sin if back else sin
    r = v[..., :rot]
    if c["pairs"]:
        p, q = r[..., 0::2], r[..., 1::2]
        r = torch.stack([p * cos - q * sin, q * cos + p * sin], -1).flatten(-2)
    else:
        p, q = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([p * cos - q * sin, q * cos + p * sin], -1)
    return torch.cat([r, v[..., rot:]], -1)


_EPS = 1e-6


def _norm_plain(s):
    c = s["case"]
    share = 1.0 / c["dim"] if c["kind"] == "rms" else 1.0
    out = {}

    def one(n):
        x, w = s[n].float(), s[n + "_weight"]
        r = torch.rsqrt(share * (x * x).sum(-1, keepdim=True) + _EPS)
        xh = x * r
        out[n + "_out"] = _rotate(xh if w is None else xh * w, s, False).to(s[n].dtype)
        if c["mode"] == "train":
            du = _rotate(s["d" + n + "_out"], s, True)
            if w is not None:
                out["d" + n + "_weight"] = (du * xh).flatten(0, 2).sum(0)
                du = du * w
            out["d" + n] = r * (du - xh * (share * (du * xh).sum(-1, keepdim=True)))

    one("q")
    one("k")
    return out


# -------------------------------------------------------------- the package
def _workspace(s, nbytes):
    """The scratch memory that a user's program keeps between calls."""
    if s.get("ws") is None:
        s["ws"] = torch.empty(max(256, nbytes), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _cu_arg(s):
    return s["cu"] if s["case"]["packed"] else None


def _conv_own(s):
    import gated_delta_rule_158_b200 as kda
    c = s["case"]
    act = kda.KDA_ACT_SILU if c["silu"] else kda.KDA_ACT_NONE
    if c["mode"] == "step":
        kda.kda_short_conv_step(s["x"], s["weight"], s["state"], s["out"], bias=s["bias"],
                                activation=act)
        return {"out": s["out"], "state": s["state"]}
    cu = _cu_arg(s)
    if s.get("ws") is None:
        _workspace(s, kda.kda_short_conv_bwd_workspace_size(
            s["x"].shape[0], s["x"].shape[1], c["channels"], c["width"],
            c["seqs"] if c["packed"] else 0) if c["mode"] == "train" else 256)
    ws = s["ws"]
    kda.kda_short_conv_fwd(s["x"], s["weight"], s["out"], ws, bias=s["bias"],
                           init_state=s["state"], cu_seqlens=cu, final_state=s.get("final"),
                           activation=act)
    out = {"out": s["out"]}
    if s["state"] is not None:
        out["final"] = s["final"]
    if c["mode"] == "train":
        grads = {"dx": s["dx"], "dweight": s["dweight"]}
        if s["bias"] is not None:
            grads["dbias"] = s["dbias"]
        if s["state"] is not None:
            grads["d_init"] = s["d_init"]
        kda.kda_short_conv_bwd(s["x"], s["weight"], s["dout"], grads, ws, bias=s["bias"],
                               init_state=s["state"], d_final=s.get("d_final"), cu_seqlens=cu,
                               activation=act)
        out.update(grads)
    return out


def _scan_own(s):
    import gated_delta_rule_158_b200 as kda
    c = s["case"]
    if c["mode"] == "step":
        kda.kda_selective_scan_step(s["x"], s["delta"], s["A"], s["B"], s["C"], s["state"],
                                    s["out"], D=s["D"], z=s["z"], delta_bias=s["delta_bias"],
                                    delta_softplus=True)
        return {"out": s["out"], "state": s["state"]}
    cu = _cu_arg(s)
    train = c["mode"] == "train"
    if s.get("ws") is None:
        shape = (s["x"].shape[0], s["x"].shape[1], c["channels"], c["dstate"], c["groups"],
                 c["seqs"] if c["packed"] else 0)
        need = kda.kda_selective_scan_fwd_workspace_size(*shape)
        if train:
            need = max(need, kda.kda_selective_scan_bwd_workspace_size(*shape))
        _workspace(s, need)
    ws = s["ws"]
    opt = dict(D=s["D"], z=s["z"], delta_bias=s["delta_bias"], delta_softplus=True,
               init_state=s["state"], cu_seqlens=cu)
    kda.kda_selective_scan_fwd(s["x"], s["delta"], s["A"], s["B"], s["C"], s["out"], ws,
                               final_state=s.get("final"), **opt)
    out = {"out": s["out"]}
    if s["state"] is not None:
        out["final"] = s["final"]
    if train:
        names = ["dx", "ddelta", "dA", "dB", "dC", "dD", "ddelta_bias"]
        names += ["dz"] if s["z"] is not None else []
        names += ["d_init"] if s["state"] is not None else []
        grads = {n: s[n] for n in names}
        kda.kda_selective_scan_bwd(s["x"], s["delta"], s["A"], s["B"], s["C"], s["dout"], grads,
                                   ws, d_final=s.get("d_final"), **opt)
        out.update(grads)
    return out


def _norm_own(s):
    import gated_delta_rule_158_b200 as kda
    c = s["case"]
    opt = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], positions=s["positions"],
               inv_freq=s["inv_freq"], eps=_EPS,
               mode=kda.KDA_NORM_RMS if c["kind"] == "rms" else kda.KDA_NORM_L2,
               rotation=kda.KDA_ROT_PAIRS if c["pairs"] else kda.KDA_ROT_HALVES)
    kda.kda_qk_norm_fwd(s["q"], s["k"], s["q_out"], s["k_out"], **opt)
    out = {"q_out": s["q_out"], "k_out": s["k_out"]}
    if c["mode"] == "train":
        names = ["dq", "dk"] + (["dq_weight", "dk_weight"] if c["weights"] else [])
        grads = {n: s[n] for n in names}
        if s.get("ws") is None:
            _workspace(s, kda.kda_qk_norm_bwd_workspace_size(
                c["tokens"], c["q_heads"], c["k_heads"], c["dim"]))
        kda.kda_qk_norm_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], grads, s["ws"], **opt)
        out.update(grads)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _conv_own, "scan": _scan_own, "norm": _norm_own}[op](state)
    return {"conv": _conv_plain, "scan": _scan_plain, "norm": _norm_plain}[op](state)


# ------------------------------------------------------------------ exact
def _exact_conv(s, case):
    """Sequence by sequence, window by window in fp64; gradients by differentiation."""
    W, train = case["width"], case["mode"] == "train"
    if case["mode"] == "step":
        x, cu = s["x"][:, None], None
    else:
        x = _flat(s["x"])[None]
        cu = s["cu"].tolist()
    w = s["weight"].double().requires_grad_(train)
    b = s["bias"].double().requires_grad_(train) if s["bias"] is not None else None
    n = case["seqs"]
    outs, finals, dxs, dis = [], [], [], []
    for i in range(n):
        xi = (x[i] if cu is None else x[0, cu[i]:cu[i + 1]]).double().requires_grad_(train)
        D = xi.shape[-1]
        s0 = s["state"][i].double() if s["state"] is not None else xi.new_zeros(W - 1, D)
        s0 = s0.detach().requires_grad_(train)
        ext = torch.cat([s0, xi])
        if xi.shape[0]:
            p = (ext.unfold(0, W, 1) * w).sum(-1)
            p = p + b if b is not None else p
            y = torch.nn.functional.silu(p) if case["silu"] else p
        else:
            y = xi
        fin = ext[ext.shape[0] - (W - 1):]
        outs.append(y.detach())
        finals.append(fin.detach())
        if train:
            loss = (y * _flat(s["dout"])[cu[i]:cu[i + 1]].double()).sum()
            if s["state"] is not None:
                loss = loss + (fin * s["d_final"][i].double()).sum()
            if loss.requires_grad:
                loss.backward()
            dxs.append(xi.grad if xi.grad is not None else torch.zeros_like(xi))
            dis.append(s0.grad if s0.grad is not None else torch.zeros_like(s0))
    if case["mode"] == "step":
        return {"out": torch.cat(outs), "state": torch.stack(finals)}
    out = {"out": torch.cat(outs).view(s["x"].shape)}
    if s["state"] is not None:
        out["final"] = torch.stack(finals)
    if train:
        out["dx"] = torch.cat(dxs).view(s["x"].shape)
        out["dweight"] = w.grad
        if b is not None:
            out["dbias"] = b.grad
        if s["state"] is not None:
            out["d_init"] = torch.stack(dis)
    return out


def _exact_scan(s, case):
    """Token by token in fp64; gradients by differentiation."""
    D, N, G = case["channels"], case["dstate"], case["groups"]
    train, step = case["mode"] == "train", case["mode"] == "step"
    n = case["seqs"]
    p = {k: s[k].double().requires_grad_(train) for k in ("A", "D", "delta_bias")}
    names = ["x", "delta", "B", "C"] + (["z"] if s["z"] is not None else [])
    if step:
        groups = [([slice(0, n)], {k: s[k].double()[:, None] for k in names})]
    elif case["packed"]:
        cu = s["cu"].tolist()
        groups = [([slice(i, i + 1)], {k: s[k][:, cu[i]:cu[i + 1]].double() for k in names})
                  for i in range(n)]
    else:
        groups = [([slice(0, n)], {k: s[k].double() for k in names})]
    outs, finals, grads, dis = [], [], {k: [] for k in names}, []
    at = 0
    for (rows,), v in groups:
        v = {k: t.detach().requires_grad_(train) for k, t in v.items()}
        S, T = v["x"].shape[:2]
        h0 = s["state"][rows].double() if s["state"] is not None else \
            torch.zeros(S, D, N, dtype=torch.float64, device=s["x"].device)
        h = h0 = h0.detach().requires_grad_(train)
        u = v["delta"] + p["delta_bias"]
        dt = torch.log1p(torch.exp(-u.abs())) + u.clamp(min=0)
        ys = []
        for xt, d, Bt, Ct in zip(*(q.unbind(1) for q in (v["x"], dt, v["B"], v["C"]))):
            Bt, Ct = Bt.repeat_interleave(D // G, 1), Ct.repeat_interleave(D // G, 1)
            h = torch.exp(d[..., None] * p["A"]) * h + (d * xt)[..., None] * Bt
            ys.append((h * Ct).sum(-1))
        y = torch.stack(ys, 1) + p["D"] * v["x"] if T else v["x"] * p["D"]
        if s["z"] is not None:
            y = y * torch.nn.functional.silu(v["z"])
        outs.append(y.detach())
        finals.append(h.detach())
        if train:
            do = s["dout"].double()
            do = do[:, at:at + T] if case["packed"] else do
            loss = (y * do).sum()
            if s["state"] is not None:
                loss = loss + (h * s["d_final"][rows].double()).sum()
            loss.backward()
            for k in names:
                grads[k].append(v[k].grad if v[k].grad is not None else torch.zeros_like(v[k]))
            dis.append(h0.grad if h0.grad is not None else torch.zeros_like(h0))
        at += T
    if step:
        return {"out": outs[0][:, 0], "state": finals[0]}
    out = {"out": torch.cat(outs, 1)}
    if s["state"] is not None:
        out["final"] = torch.cat(finals)
    if train:
        for k in names:
            out["d" + k] = torch.cat(grads[k], 1)
        for k in ("A", "D", "delta_bias"):
            out["d" + k] = p[k].grad
        if s["state"] is not None:
            out["d_init"] = torch.cat(dis)
    return out


def _exact_norm(s, case):
    """Rows scaled in fp64 and turned as complex numbers; gradients by differentiation."""
    train, rot, d = case["mode"] == "train", case["rot"], case["dim"]
    out = {}
    for n in ("q", "k"):
        x = s[n].double().requires_grad_(train)
        w = s[n + "_weight"]
        w = torch.ones(d, dtype=torch.float64, device=x.device) if w is None else w.double()
        w = w.detach().requires_grad_(train)
        size = x.pow(2).mean(-1) if case["kind"] == "rms" else x.pow(2).sum(-1)
        y = x / (size + _EPS).sqrt()[..., None] * w
        if rot:
            ang = s["positions"].double()[0, :, None] * s["inv_freq"].double()
            turn = torch.polar(torch.ones_like(ang), ang)[None, :, None]
            r = y[..., :rot]
            r = r.unflatten(-1, (rot // 2, 2)) if case["pairs"] else \
                r.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            r = torch.view_as_real(torch.complex(r[..., 0], r[..., 1]) * turn)
            r = r.flatten(-2) if case["pairs"] else r.transpose(-1, -2).flatten(-2)
            y = torch.cat([r, y[..., rot:]], -1)
        out[n + "_out"] = y.detach()
        if train:
            y.backward(s["d" + n + "_out"].double())
            out["d" + n] = x.grad
            if s[n + "_weight"] is not None:
                out["d" + n + "_weight"] = w.grad
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "scan" and case["mode"] == "train":
        # several fp64 states are held for every token
        if case["tokens"] > 16384:
            return None
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](s, case)
