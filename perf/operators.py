"""Plain forms, exact forms and measured cases of the training operators that
surround the row normalisations: group normalisation with an activation and
dropout on channels-last tensors, dropout from a counter-based generator, and
dropout + residual add + RMSNorm / LayerNorm.

`own` selects what run() calls: the plain form (elementary torch operations
in 32 bits) or the library's entry points.

The dropout mask is a function of (seed, offset, element index): block i of
eight consecutive elements takes the four 32-bit outputs of Philox4x32-10
(Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3",
SC 2011) at counter (i, offset) under the key `seed`; element e of the block
reads the 16-bit half e (the low half of word e / 2 first) and is kept when
that is at least T = p * 2^16 (to the nearest integer); kept elements are
multiplied by 2^16 / (2^16 - T), dropped ones become 0.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
RMS, LAYER = 0, 1


def listed():
    return [
        # one sample at the lowest resolution of a convolutional denoiser: the latency case
        dict(name="group_fwd_step", op="group_fwd", dtype="bf16", B=1, S=64, C=1280, G=32,
             act="silu", p=0.0),
        # a training batch at 64 x 64 positions, groups of 10 channels (not a 16-byte multiple)
        dict(name="group_fwd_train", op="group_fwd", dtype="bf16", B=8, S=4096, C=320, G=32,
             act="silu", p=0.0),
        # an image decoder's last blocks: one sample of 512 x 512 positions
        dict(name="group_fwd_image", op="group_fwd", dtype="fp16", B=1, S=262144, C=256, G=32,
             act="silu", p=0.0),
        # ragged positions (37 x 41) and groups of 14 channels in 32 bits, no activation
        dict(name="group_fwd_odd", op="group_fwd", dtype="fp32", B=3, S=1517, C=168, G=12,
             act="none", p=0.0),
        # the second half of a residual block in training: norm, SiLU, dropout
        dict(name="group_bwd_train", op="group_bwd", dtype="bf16", B=16, S=1024, C=640, G=32,
             act="silu", p=0.1),
        # training at 128 x 128 positions
        dict(name="group_bwd_large", op="group_bwd", dtype="bf16", B=4, S=16384, C=512, G=32,
             act="silu", p=0.0),
        # small ragged backward, eight channels per group
        dict(name="group_bwd_odd", op="group_bwd", dtype="fp16", B=2, S=221, C=88, G=11,
             act="gelu", p=0.0),
        # dropout of a small 32-bit tensor of odd length
        dict(name="dropout_small", op="dropout", dtype="fp32", M=257, N=333, p=0.5),
        # dropout of the activations of the LayerNorm workload (the backward is the same call)
        dict(name="dropout_large", op="dropout", dtype="bf16", M=32768, N=4096, p=0.1),
        # the small RMSNorm workload behind a dropped-out residual branch
        dict(name="add_fwd_small", op="add_fwd", mode=RMS, M=256, N=1024, p=0.1),
        # the LayerNorm workload behind a dropped-out residual branch, both directions
        dict(name="add_fwd_layer", op="add_fwd", mode=LAYER, M=32768, N=4096, p=0.1),
        dict(name="add_bwd_layer", op="add_bwd", mode=LAYER, M=32768, N=4096, p=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["group_fwd", "group_bwd", "dropout", "add_fwd", "add_bwd"])
    if op in ("group_fwd", "group_bwd"):
        # group counts and channels per group that make C a multiple of 8
        G = rng.choice([1, 4, 8, 16, 32, 32, 32])
        D = rng.choice([4, 8, 10, 14, 16, 20, 32, 40, 64])
        while (G * D) % 8:
            D += 2
        C = G * D
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        S = _log(rng, 1, 262144)
        most = (1 << 25) if op == "group_bwd" or dtype == "fp32" else (1 << 26)
        S = max(1, min(S, most // C))
        B = _log(rng, 1, max(1, min(64, most // (C * S))))
        return dict(op=op, dtype=dtype, B=B, S=S, C=C, G=G,
                    act=rng.choice(["none", "silu", "silu", "gelu"]),
                    p=rng.choice([0.0, 0.0, 0.1, 0.25]))
    if op == "dropout":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        N = _log(rng, 1, 16384)
        M = _log(rng, 1, max(1, (1 << (25 if dtype == "fp32" else 26)) // N))
        return dict(op=op, dtype=dtype, M=M, N=N, p=rng.choice([0.05, 0.1, 0.25, 0.5]))
    N = 8 * _log(rng, 8, 2048)
    M = _log(rng, 1, max(1, (1 << 26) // N))
    return dict(op=op, mode=rng.choice([RMS, LAYER]), M=M, N=N, p=rng.choice([0.05, 0.1, 0.25]))


EPS = 1e-5


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    f32 = dict(dtype=torch.float32, device=dev, generator=g)
    s = dict(case)
    s["seed"] = (0x9E3779B97F4A7C15 * (seed + 1)) % (1 << 63)
    s["offset"] = 3 + seed % 1000
    if case["op"] in ("group_fwd", "group_bwd"):
        B, S, C, G = case["B"], case["S"], case["C"], case["G"]
        dt = DT[case["dtype"]]
        # activations of a convolution: a mean per channel and noise around it
        x = torch.randn(B, S, C, **f32)
        x += 0.5 * torch.randn(C, **f32)
        s["x"] = x = x.to(dt)
        s["gamma"] = (1.0 + 0.1 * torch.randn(C, **f32)).to(dt)
        s["beta"] = (0.1 * torch.randn(C, **f32)).to(dt)
        if case["op"] == "group_bwd":
            s["dy"] = torch.randn(B, S, C, **f32).to(dt)
            xg = x.view(B, S, G, C // G)
            mean = xg.sum((1, 3), dtype=torch.float64) / (S * (C // G))
            d = xg.double() - mean.view(B, 1, G, 1)
            s["mean"] = mean.float()
            s["rstd"] = ((d * d).mean((1, 3)) + EPS).rsqrt().float()
    elif case["op"] == "dropout":
        s["x"] = torch.randn(case["M"], case["N"], **f32).to(DT[case["dtype"]])
    else:
        M, N, dt = case["M"], case["N"], torch.bfloat16
        s["gamma"] = (1.0 + 0.1 * torch.randn(N, **f32)).to(dt)
        s["beta"] = (0.1 * torch.randn(N, **f32)).to(dt) if case["mode"] == LAYER else None
        h = (torch.randn(M, N, **f32) + 0.5 * torch.randn(N, **f32)).to(dt)
        if case["op"] == "add_fwd":
            s["x"], s["r"] = torch.randn(M, N, **f32).to(dt), h
        else:
            s["h"] = h
            s["dy"], s["dh"] = torch.randn(M, N, **f32).to(dt), torch.randn(M, N, **f32).to(dt)
            hd = h.double()
            mean = hd.mean(1) if case["mode"] == LAYER else torch.zeros(M, dtype=torch.float64,
                                                                        device=dev)
            hd -= mean[:, None]
            s["rstd"] = (hd.square_().mean(1) + EPS).rsqrt().float()
            s["mean"] = mean.float() if case["mode"] == LAYER else None
    return s


# ------------------------------------------------------------- plain forms
def _keep(n, p, seed, offset, dev):
    """Truth value per element (kept), and the factor of kept elements."""
    T = int(p * 65536 + 0.5)
    low = 0xFFFFFFFF
    i = torch.arange((n + 7) // 8, dtype=torch.int64, device=dev)
    c0, c1 = i & low, i >> 32
    c2, c3 = torch.full_like(i, offset & low), torch.full_like(i, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64-bit products (bits, whatever the sign)
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    w = torch.stack((c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16,
                     c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16), 1)
    return (w >= T).view(-1)[:n], 65536.0 / (65536 - T)


def _drop(v, s):
    """Dropout of the 32-bit tensor v."""
    if s["p"] == 0.0:
        return v
    keep, scale = _keep(v.numel(), s["p"], s["seed"], s["offset"], v.device)
    return torch.where(keep.view(v.shape), v * scale, torch.zeros((), device=v.device))


def _act_arg(z, act):
    """k(z) with act(z) = z * sigmoid(k(z)), and its derivative."""
    if act == "silu":
        return z, 1.0
    c = 2.0 * math.sqrt(2.0 / math.pi)  # GELU, tanh form
    return c * (z + 0.044715 * z * z * z), c * (1.0 + 3 * 0.044715 * z * z)


def _sigmoid(k):
    return 1.0 / (1.0 + torch.exp(-k))


def _group_fwd_plain(s):
    x = s["x"].float()
    B, S, C, G = s["B"], s["S"], s["C"], s["G"]
    xg = x.view(B, S, G, C // G)
    mean = xg.mean((1, 3), keepdim=True)
    d = xg - mean
    rstd = 1.0 / torch.sqrt((d * d).mean((1, 3), keepdim=True) + EPS)
    z = (d * rstd).view(B, S, C) * s["gamma"].float() + s["beta"].float()
    if s["act"] != "none":
        z = z * _sigmoid(_act_arg(z, s["act"])[0])
    return _drop(z, s).to(s["x"].dtype), rstd.view(B, G), mean.view(B, G)


def _group_bwd_plain(s):
    dt = s["x"].dtype
    B, S, C, G = s["B"], s["S"], s["C"], s["G"]
    gamma, beta = s["gamma"].float(), s["beta"].float()
    rstd = s["rstd"].view(B, 1, G, 1)
    xhat = ((s["x"].float().view(B, S, G, C // G) - s["mean"].view(B, 1, G, 1)) * rstd).view(B, S, C)
    dz = _drop(s["dy"].float(), s)
    if s["act"] != "none":
        z = xhat * gamma + beta
        k, dk = _act_arg(z, s["act"])
        sg = _sigmoid(k)
        dz = dz * (sg + z * sg * (1.0 - sg) * dk)
    dgamma, dbeta = (dz * xhat).sum((0, 1)), dz.sum((0, 1))
    g = (dz * gamma).view(B, S, G, C // G)
    xh = xhat.view(B, S, G, C // G)
    a, c = g.mean((1, 3), keepdim=True), (g * xh).mean((1, 3), keepdim=True)
    dx = rstd * (g - a - xh * c)
    return dx.view(B, S, C).to(dt), dgamma, dbeta


def _norm_stats(hf, mode):
    mean = hf.mean(1, keepdim=True) if mode == LAYER else None
    d = hf - mean if mode == LAYER else hf
    return d, 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS), mean


def _add_fwd_plain(s):
    h = (s["r"].float() + _drop(s["x"].float(), s)).to(torch.bfloat16)
    d, rstd, mean = _norm_stats(h.float(), s["mode"])
    y = d * rstd * s["gamma"].float()
    if s["mode"] == LAYER:
        y = y + s["beta"].float()
    return h, y.to(torch.bfloat16), rstd.view(-1), None if mean is None else mean.view(-1)


def _add_bwd_plain(s):
    layer = s["mode"] == LAYER
    rstd = s["rstd"][:, None]
    d = s["h"].float() - s["mean"][:, None] if layer else s["h"].float()
    xhat, dy = d * rstd, s["dy"].float()
    g = dy * s["gamma"].float()
    t = g - xhat * (g * xhat).mean(1, keepdim=True)
    if layer:
        t = t - g.mean(1, keepdim=True)
    t = rstd * t + s["dh"].float()
    return (_drop(t, s).to(torch.bfloat16), t.to(torch.bfloat16), (dy * xhat).sum(0),
            dy.sum(0) if layer else None)


def run(state):
    s = state
    op = s["op"]
    if own:
        import memory_bound_normalization_rmsnorm_gb300 as gb

        rng = dict(p=s["p"], seed=s["seed"], offset=s["offset"])
        if op == "group_fwd":
            return gb.norm_group_fwd(s["x"], s["gamma"], s["beta"], s["G"], EPS, s["act"], **rng)
        if op == "group_bwd":
            return gb.norm_group_bwd(s["dy"], s["x"], s["gamma"], s["beta"], s["rstd"], s["mean"],
                                     s["G"], s["act"], **rng)
        if op == "dropout":
            return gb.norm_dropout(s["x"], **rng)
        if op == "add_fwd":
            return gb.norm_dropout_add_fwd(s["x"], s["r"], s["gamma"], s["beta"], EPS, s["mode"],
                                           **rng)
        return gb.norm_dropout_add_bwd(s["dy"], s["dh"], s["h"], s["gamma"], s["rstd"], s["mean"],
                                       s["mode"], **rng)
    if op == "group_fwd":
        return _group_fwd_plain(s)
    if op == "group_bwd":
        return _group_bwd_plain(s)
    if op == "dropout":
        return _drop(s["x"].float(), s).to(s["x"].dtype)
    return _add_fwd_plain(s) if op == "add_fwd" else _add_bwd_plain(s)


def work(case):
    """Each input read once, each output written once; the arithmetic of the
    definition (a multiply, an add or an exponential each count one)."""
    op = case["op"]
    drop = 0 if case["p"] == 0.0 else 2
    if op in ("group_fwd", "group_bwd"):
        n, es = case["B"] * case["S"] * case["C"], 4 if case["dtype"] == "fp32" else 2
        stats, act = 8 * case["B"] * case["G"], 0 if case["act"] == "none" else 5
        if op == "group_fwd":
            return {"bytes": 2 * n * es + 2 * case["C"] * es + stats, "flops": n * (8 + act + drop)}
        return {"bytes": 3 * n * es + case["C"] * (2 * es + 8) + stats,
                "flops": n * (13 + 2 * act + drop)}
    n = case["M"] * case["N"]
    if op == "dropout":
        return {"bytes": 2 * n * (4 if case["dtype"] == "fp32" else 2), "flops": 2 * n}
    k = 2 if case["mode"] == LAYER else 1
    if op == "add_fwd":
        return {"bytes": 8 * n + 2 * k * case["N"] + 4 * k * case["M"], "flops": 11 * n}
    return {"bytes": 10 * n + case["N"] * (2 + 4 * k) + 4 * k * case["M"], "flops": 15 * n}


# ------------------------------------------------ the definitions in 64 bits
def _words(blocks, seed, offset):
    """Philox4x32-10 at counters (0 .. blocks-1, offset): uint32 [blocks, 4]."""
    m = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    x = [np.arange(blocks, dtype=np.uint64), None,
         np.full(blocks, offset % (1 << 32), np.uint64), np.full(blocks, offset >> 32, np.uint64)]
    x[1] = x[0] >> sh
    x[0] = x[0] & m
    key = [seed % (1 << 32), seed >> 32]
    for r in range(10):
        hi0, lo0 = np.divmod(x[0] * np.uint64(0xD2511F53), np.uint64(1 << 32))
        hi1, lo1 = np.divmod(x[2] * np.uint64(0xCD9E8D57), np.uint64(1 << 32))
        kr = [np.uint64((key[0] + r * 0x9E3779B9) % (1 << 32)),
              np.uint64((key[1] + r * 0xBB67AE85) % (1 << 32))]
        x = [hi1 ^ x[1] ^ kr[0], lo1, hi0 ^ x[3] ^ kr[1], lo0]
    return np.stack([v.astype(np.uint32) for v in x], axis=1)


def _factor64(shape, s):
    """Per element 0 or 2^16 / (2^16 - T), in float64."""
    n = int(np.prod(shape))
    T = round(s["p"] * 65536)
    halves = np.ascontiguousarray(_words((n + 7) // 8, s["seed"], s["offset"])).astype("<u4")
    halves = halves.view("<u2").reshape(-1)[:n].astype(np.int32)
    kept = torch.from_numpy(halves).to("cuda") >= T
    return kept.double().mul_(65536.0 / (65536.0 - T)).view(shape)


def _act64(z, act):
    if act == "silu":
        return torch.nn.functional.silu(z)
    if act == "gelu":
        return torch.nn.functional.gelu(z, approximate="tanh")
    return z


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        x = s["x"].double()
        return x * _factor64(x.shape, s)
    if op in ("group_fwd", "group_bwd"):
        grads = op == "group_bwd"
        gamma = s["gamma"].double().requires_grad_(grads)
        beta = s["beta"].double().requires_grad_(grads)
        x = s["x"].double().requires_grad_(grads)
        xc = x.reshape(s["B"], s["S"], s["G"], -1)
        mean = xc.mean((1, 3))
        var = xc.var((1, 3), unbiased=False) if xc.shape[1] * xc.shape[3] > 1 else 0.0 * mean
        rstd = (var + EPS) ** -0.5
        xhat = (xc - mean[:, None, :, None]) * rstd[:, None, :, None]
        y = _act64(xhat.reshape(x.shape) * gamma + beta, s["act"])
        if case["p"]:
            y = y * _factor64(y.shape, s)
        if not grads:
            return y, rstd, mean
        return torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
    layer = case["mode"] == LAYER
    fac = _factor64((s["M"], s["N"]), s)
    if op == "add_fwd":
        h = (s["r"].double() + s["x"].double() * fac).to(torch.bfloat16)
    else:
        h = s["h"]
    hd = h.double().requires_grad_(op == "add_bwd")
    gamma = s["gamma"].double().requires_grad_(op == "add_bwd")
    beta = s["beta"].double().requires_grad_(op == "add_bwd") if layer else None
    mean = hd.mean(1) if layer else None
    c = hd - mean[:, None] if layer else hd
    rstd = (c.square().mean(1) + EPS) ** -0.5
    y = c * rstd[:, None] * gamma
    if layer:
        y = y + beta
    if op == "add_fwd":
        return h.double(), y, rstd, mean
    grads = torch.autograd.grad(y, (hd, gamma, beta) if layer else (hd, gamma), s["dy"].double())
    total = grads[0] + s["dh"].double()
    return total * fac, total, grads[1], grads[2] if layer else None
