"""Plain forms, exact forms and measured cases of the operators between the
normalisations of a pre-norm transformer block: the linear layer with bias,
activation and residual in its epilogue, and the normalisation and rotation
(rotary positions of one or several axes) of query and key heads.

`own` selects what run() calls: the plain form (elementary torch operations
in 32 bits) or the library's entry points.

Linear: z = x W^T + b, y = r + act(z) with x [M, K], W [N, K].  Its backward
pass takes dy and z: dz = dy act'(z), db = column sums of dz, dx = dz W,
dW = dz^T x (the gradient of r is dy).

Rotation: pair p of a head's first `rd` elements (p and p + rd / 2, or 2p and
2p + 1) turns by pos[axis of p] * inv_freq[p]; before it each head row of D
elements is normalised (RMSNorm or LayerNorm over D) where the case has a mode.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
RMS, LAYER = 0, 1
EPS = 1e-6


def listed():
    return [
        # one token through a projection back to the residual stream: serving, latency counts
        dict(name="linear_token", op="linear_fwd", dtype="bf16", M=1, K=4096, N=4096, act="none",
             bias=True, res=True, z=False),
        # a batch of sequences decoding side by side, up-projection
        dict(name="linear_decode", op="linear_fwd", dtype="bf16", M=48, K=4096, N=16384, act="silu",
             bias=True, res=False, z=False),
        # a training batch through the up-projection of a block, z kept for the backward pass
        dict(name="linear_up_train", op="linear_fwd", dtype="bf16", M=8192, K=4096, N=16384,
             act="gelu", bias=True, res=False, z=True),
        # the down-projection of a prompt, added to the residual stream
        dict(name="linear_down_prompt", op="linear_fwd", dtype="bf16", M=2048, K=8192, N=5120,
             act="none", bias=False, res=True, z=False),
        # sizes that no vector width divides
        dict(name="linear_odd", op="linear_fwd", dtype="fp16", M=777, K=1234, N=999, act="silu",
             bias=True, res=True, z=True),
        # gradients of the up-projection
        dict(name="linear_bwd_train", op="linear_bwd", dtype="bf16", M=4096, K=4096, N=16384,
             act="gelu", bias=True),
        # gradients of a small ragged batch
        dict(name="linear_bwd_odd", op="linear_bwd", dtype="fp16", M=531, K=648, N=1001, act="none",
             bias=True),
        # one token of each of four sequences: 32 query and 8 key heads, three axes
        dict(name="rope_token", op="rope_fwd", dtype="bf16", T=4, Hq=32, Hk=8, D=128, rd=128,
             axes=3, mode="rms", inter=False, per_axis=False, packed=True),
        # a video prompt
        dict(name="rope_prompt", op="rope_fwd", dtype="bf16", T=32768, Hq=32, Hk=8, D=128, rd=128,
             axes=3, mode="rms", inter=False, per_axis=False, packed=True),
        # image patches: a frequency ladder for each of two axes, neighbours as pairs, LayerNorm
        dict(name="rope_image", op="rope_fwd", dtype="fp32", T=5476, Hq=16, Hk=16, D=80, rd=80,
             axes=2, mode="layer", inter=True, per_axis=True, packed=False),
        # training on video: gradients of q, k and of both scales
        dict(name="rope_bwd_train", op="rope_bwd", dtype="bf16", T=16384, Hq=32, Hk=8, D=128, rd=128,
             axes=3, mode="rms", inter=False, per_axis=False, packed=True),
        # part of each head turns, small ragged batch, no norm
        dict(name="rope_bwd_odd", op="rope_bwd", dtype="fp16", T=333, Hq=12, Hk=4, D=72, rd=36,
             axes=1, mode="none", inter=False, per_axis=False, packed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_fwd", "linear_bwd", "rope_fwd", "rope_bwd"])
    if op.startswith("linear"):
        step = rng.choice([64, 64, 8, 1])
        K = max(step, _log(rng, 64, 16384) // step * step)
        N = max(step, _log(rng, 64, 16384) // step * step)
        most = 8192 * 4096 * 16384 // (2 if op == "linear_bwd" else 1)
        M = _log(rng, 1, max(1, min(16384, most // (K * N))))
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), M=M, K=K, N=N,
                 act=rng.choice(["none", "silu", "gelu"]), bias=rng.choice([True, False]))
        if op == "linear_fwd":
            c.update(res=rng.choice([True, False]), z=rng.choice([True, False]))
        return c
    D = rng.choice([32, 64, 72, 80, 96, 128, 128, 256])
    rd = rng.choice([D, D, D, D // 2])
    Hk = rng.choice([1, 2, 4, 8, 12])
    Hq = Hk * rng.choice([1, 2, 4])
    T = _log(rng, 1, min(32768, 32768 * 40 * 128 // (2 if op == "rope_bwd" else 1) // ((Hq + Hk) * D)))
    axes = rng.choice([1, 2, 3])
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), T=T, Hq=Hq, Hk=Hk, D=D,
                rd=rd, axes=axes, mode=rng.choice(["none", "rms", "rms", "layer"]),
                inter=rng.choice([True, False]), per_axis=axes > 1 and rng.choice([True, False]),
                packed=rng.choice([True, False]))


def _sections(pairs, axes):
    """Pairs per axis: halves, or 2 : 3 : 3 for time, height and width."""
    if axes == 1:
        return (pairs,)
    if axes == 2:
        return (pairs - pairs // 2, pairs // 2)
    s = pairs * 3 // 8
    return (pairs - 2 * s, s, s)


def _inv_freq(rd, sections, per_axis):
    """base^(-2 i / rd) over all pairs, or a ladder of its own for each axis."""
    f = []
    if per_axis:
        for n in sections:
            f += [10000.0 ** (-i / n) for i in range(n)]
    else:
        f = [10000.0 ** (-2.0 * i / rd) for i in range(rd // 2)]
    return f


def _positions(T, axes, g, dev):
    """Token positions [axes, T]: a stretch of text (all axes alike), then frames of a grid."""
    start = int(torch.randint(0, 1 << 20, (1,), device=dev, generator=g))
    i = torch.arange(T, device=dev)
    if axes == 1:
        return i + start
    text = T // 8
    j = i - text
    side = max(1, int(math.isqrt(max(1, (T - text) // 4))))
    grid = [j // (side * side), j // side % side, j % side][3 - axes:]
    return torch.stack([start + torch.where(i < text, i, text + c) for c in grid])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    f32 = dict(dtype=torch.float32, device=dev, generator=g)
    s = dict(case)
    dt = DT[case["dtype"]]
    if case["op"].startswith("linear"):
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = torch.randn(M, K, **f32).to(dt)
        s["w"] = (torch.randn(N, K, **f32) / math.sqrt(K)).to(dt)
        if case["op"] == "linear_fwd":
            s["b"] = (0.1 * torch.randn(N, **f32)).to(dt) if case["bias"] else None
            s["r"] = torch.randn(M, N, **f32).to(dt) if case["res"] else None
        else:
            s["dy"] = torch.randn(M, N, **f32).to(dt)
            # what the forward kept: unit variance, like x W^T here
            s["zs"] = torch.randn(M, N, **f32).to(dt) if case["act"] != "none" else None
        return s
    T, Hq, Hk, D, rd = case["T"], case["Hq"], case["Hk"], case["D"], case["rd"]

    def heads():
        """q and k: views of one projection's rows (query, key and value heads), or tensors."""
        if case["packed"]:
            rows = torch.randn(T, (Hq + 2 * Hk) * D, **f32).to(dt)
            return (rows[:, :Hq * D].view(T, Hq, D),
                    rows[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D))
        return torch.randn(T, Hq, D, **f32).to(dt), torch.randn(T, Hk, D, **f32).to(dt)

    s["q"], s["k"] = heads()
    if case["op"] == "rope_bwd":
        s["dyq"] = torch.randn(T, Hq, D, **f32).to(dt)
        s["dyk"] = torch.randn(T, Hk, D, **f32).to(dt)
    norm, layer = case["mode"] != "none", case["mode"] == "layer"
    s["gq"] = (1.0 + 0.1 * torch.randn(D, **f32)).to(dt) if norm else None
    s["gk"] = (1.0 + 0.1 * torch.randn(D, **f32)).to(dt) if norm else None
    s["bq"] = (0.1 * torch.randn(D, **f32)).to(dt) if layer else None
    s["bk"] = (0.1 * torch.randn(D, **f32)).to(dt) if layer else None
    s["sections"] = _sections(rd // 2, case["axes"])
    s["pos"] = _positions(T, case["axes"], g, dev)
    s["inv_freq"] = torch.tensor(_inv_freq(rd, s["sections"], case["per_axis"]), device=dev,
                                 dtype=torch.float64)
    return s


# ------------------------------------------------------------- plain forms
def _act_parts(z, act):
    """k(z) with act(z) = z * sigmoid(k(z)), and its derivative."""
    if act == "silu":
        return z, 1.0
    c = 2.0 * math.sqrt(2.0 / math.pi)  # GELU, tanh form
    return c * (z + 0.044715 * z * z * z), c * (1.0 + 3 * 0.044715 * z * z)


def _sigmoid(k):
    return 1.0 / (1.0 + torch.exp(-k))


def _linear_fwd_plain(s):
    dt = s["x"].dtype
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = z if s["act"] == "none" else z * _sigmoid(_act_parts(z, s["act"])[0])
    if s["r"] is not None:
        y = y + s["r"].float()
    return (y.to(dt), z.to(dt)) if s["z"] else y.to(dt)


def _linear_bwd_plain(s):
    dt = s["x"].dtype
    dz = s["dy"].float()
    if s["act"] != "none":
        z = s["zs"].float()
        k, dk = _act_parts(z, s["act"])
        sg = _sigmoid(k)
        dz = dz * (sg + z * sg * (1.0 - sg) * dk)
    dx = dz @ s["w"].float()
    dw = dz.t() @ s["x"].float()
    return dx.to(dt), dw.to(dt), dz.sum(0) if s["bias"] else None


def _angles(s):
    """cos and sin [T, 1, rd / 2]; the angles in 64 bits (positions reach 2^20 and more)."""
    pos = s["pos"] if s["axes"] > 1 else s["pos"][None]
    n = torch.tensor(s["sections"], device=pos.device)
    axis = torch.repeat_interleave(torch.arange(s["axes"], device=pos.device), n,
                                   output_size=s["rd"] // 2)
    a = pos[axis].t().double() * s["inv_freq"]
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _split(v, s):
    """The two elements of each pair, and the elements that do not turn."""
    rd = s["rd"]
    if s["inter"]:
        return v[..., 0:rd:2], v[..., 1:rd:2], v[..., rd:]
    return v[..., :rd // 2], v[..., rd // 2:rd], v[..., rd:]


def _join(a, b, rest, s):
    if s["inter"]:
        t = torch.stack((a, b), -1).flatten(-2)
        return torch.cat((t, rest), -1)
    return torch.cat((a, b, rest), -1)


def _norm_parts(v, mode):
    d = v - v.mean(-1, keepdim=True) if mode == "layer" else v
    return d, 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)


def _rope_fwd_plain(s):
    cos, sin = _angles(s)

    def one(x, gamma, beta):
        v = x.float()
        if gamma is not None:
            d, rstd = _norm_parts(v, s["mode"])
            v = d * rstd * gamma.float()
            if beta is not None:
                v = v + beta.float()
        a, b, rest = _split(v, s)
        return _join(a * cos - b * sin, b * cos + a * sin, rest, s).to(x.dtype)

    return one(s["q"], s["gq"], s["bq"]), one(s["k"], s["gk"], s["bk"])


def _rope_bwd_plain(s):
    cos, sin = _angles(s)

    def one(dy, x, gamma):
        a, b, rest = _split(dy.float(), s)
        dn = _join(a * cos + b * sin, b * cos - a * sin, rest, s)
        if gamma is None:
            return dn.to(x.dtype), None, None
        d, rstd = _norm_parts(x.float(), s["mode"])
        xhat = d * rstd
        g = dn * gamma.float()
        t = g - xhat * (g * xhat).mean(-1, keepdim=True)
        if s["mode"] == "layer":
            t = t - g.mean(-1, keepdim=True)
        return ((rstd * t).to(x.dtype), (dn * xhat).sum((0, 1)),
                dn.sum((0, 1)) if s["mode"] == "layer" else None)

    dq, dgq, dbq = one(s["dyq"], s["q"], s["gq"])
    dk, dgk, dbk = one(s["dyk"], s["k"], s["gk"])
    return dq, dk, dgq, dgk, dbq, dbk


def run(state):
    s = state
    op = s["op"]
    if own:
        import memory_bound_normalization_rmsnorm_gb300 as gb

        if op == "linear_fwd":
            y, z = gb.norm_linear_fwd(s["x"], s["w"], s["b"], s["r"], s["act"], want_z=s["z"])
            return (y, z) if s["z"] else y
        if op == "linear_bwd":
            return gb.norm_linear_bwd(s["dy"], s["x"], s["w"], s["zs"], s["act"],
                                      want_dbias=s["bias"])
        mode = LAYER if s["mode"] == "layer" else RMS
        how = dict(sections=s["sections"], interleaved=s["inter"])
        if op == "rope_fwd":
            return gb.norm_rope_fwd(s["q"], s["k"], s["pos"], s["inv_freq"], s["gq"], s["gk"],
                                    s["bq"], s["bk"], EPS, mode, **how)
        return gb.norm_rope_bwd(s["dyq"], s["dyk"], s["q"], s["k"], s["pos"], s["inv_freq"],
                                s["gq"], s["gk"], EPS, mode, **how)
    if op == "linear_fwd":
        return _linear_fwd_plain(s)
    if op == "linear_bwd":
        return _linear_bwd_plain(s)
    return _rope_fwd_plain(s) if op == "rope_fwd" else _rope_bwd_plain(s)


def work(case):
    """Each input read once, each output written once; the arithmetic of the
    definition (a multiply, an add or an exponential each count one)."""
    es = 4 if case["dtype"] == "fp32" else 2
    op = case["op"]
    if op.startswith("linear"):
        M, K, N = case["M"], case["K"], case["N"]
        act = 0 if case["act"] == "none" else 5
        if op == "linear_fwd":
            wide = 1 + case["res"] + case["z"]
            return {"bytes": es * (M * K + N * K + wide * M * N + N * case["bias"]),
                    "flops": 2 * M * N * K + M * N * (case["bias"] + case["res"] + act)}
        wide = 2 if act else 1
        return {"bytes": es * (2 * M * K + 2 * N * K + wide * M * N) + 4 * N * case["bias"],
                "flops": 4 * M * N * K + M * N * (case["bias"] + 2 * act)}
    T, D, rd = case["T"], case["D"], case["rd"]
    rows = T * (case["Hq"] + case["Hk"])
    norm = {"none": 0, "rms": 4, "layer": 7}[case["mode"]]
    params = {"none": 0, "rms": 1, "layer": 2}[case["mode"]] * 2 * D
    fixed = 8 * T * case["axes"] + 4 * rd
    if op == "rope_fwd":
        return {"bytes": es * (2 * rows * D + params) + fixed, "flops": rows * (3 * rd + norm * D)}
    moved = 2 if case["mode"] == "none" else 3
    return {"bytes": es * (moved * rows * D + (2 * D if norm else 0)) + 4 * params + fixed,
            "flops": rows * (3 * rd + (2 * norm + 3) * D)}


# ------------------------------------------------ the definitions in 64 bits
def _act64(z, act):
    if act == "silu":
        return torch.nn.functional.silu(z)
    if act == "gelu":
        return torch.nn.functional.gelu(z, approximate="tanh")
    return z


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear_fwd":
        b = None if s["b"] is None else s["b"].double()
        z = torch.nn.functional.linear(s["x"].double(), s["w"].double(), b)
        y = _act64(z, s["act"])
        if s["r"] is not None:
            y = s["r"].double() + y
        return (y, z) if s["z"] else y
    if op == "linear_bwd":
        dz = s["dy"].double()
        if s["zs"] is not None:
            z = s["zs"].double().requires_grad_()
            dz, = torch.autograd.grad(_act64(z, s["act"]), z, dz)
        return (torch.mm(dz, s["w"].double()), torch.mm(dz.t(), s["x"].double()),
                dz.sum(0) if s["bias"] else None)
    T, D, rd, grads = s["T"], s["D"], s["rd"], op == "rope_bwd"
    pos = s["pos"].reshape(s["axes"], T).double()
    turn = torch.cat([pos[a][:, None] * f[None] for a, f in
                      enumerate(torch.split(s["inv_freq"], s["sections"]))], 1)
    turn = torch.polar(torch.ones_like(turn), turn)[:, None]

    def one(x, gamma, beta, dy):
        x = x.double().requires_grad_(grads)
        p = [None if t is None else t.double().requires_grad_(grads) for t in (gamma, beta)]
        if grads and s["mode"] == "layer":
            p[1] = torch.zeros(D, dtype=torch.float64, device=x.device, requires_grad=True)
        v = x
        if gamma is not None and s["mode"] == "layer":
            v = torch.nn.functional.layer_norm(x, (D,), p[0], p[1], EPS)
        elif gamma is not None:
            v = x * (x.square().mean(-1, keepdim=True) + EPS) ** -0.5 * p[0]
        head = v[..., :rd]
        if s["inter"]:
            c = torch.view_as_complex(head.reshape(T, -1, rd // 2, 2).contiguous()) * turn
            head = torch.view_as_real(c).flatten(-2)
        else:
            c = torch.complex(head[..., :rd // 2], head[..., rd // 2:]) * turn
            head = torch.cat((c.real, c.imag), -1)
        y = torch.cat((head, v[..., rd:]), -1)
        if not grads:
            return y
        wrt = [t for t in (x, *p) if t is not None]
        got = list(torch.autograd.grad(y, wrt, dy.double()))
        return got + [None] * (3 - len(got))

    if not grads:
        return one(s["q"], s["gq"], s["bq"], None), one(s["k"], s["gk"], s["bk"], None)
    dq, dgq, dbq = one(s["q"], s["gq"], None, s["dyq"])
    dk, dgk, dbk = one(s["k"], s["gk"], None, s["dyk"])
    return dq, dk, dgq, dgk, dbq, dbk
