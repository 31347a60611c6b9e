"""The block operators as they are measured: channel norm, block residual and
counter dropout, in plain torch operations and through the library.

A block around a WTConv mixer is

    u   = norm(mixer(x))                       channel norm, planar in, channels-last out
    h   = linear(dropout(gelu(linear(u))))     the MLP on channels-last rows
    out = s * x + g * D(norm(h))               block residual, channels-last h, planar x and out

with the channel norm over the C channels of each pixel (or token)

    z = (h - mean) / sqrt(var + eps)  (layer)  or  h / sqrt(mean(h^2) + eps)  (rms),  v = z * weight + bias,

and the dropout D (elements, or whole samples) from Philox4x32-10 (Salmon,
Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011):
counter (group, site, offset low, offset high), key (seed low, seed high);
group = row * ceil(C / 8) + c // 8 for row = (b * H + i) * W + j; element c
takes 16 of the group's 128 bits (word (c % 8) // 2, its low half for even c)
and is kept when they are at least T = round(65536 p), then scaled by
65536 / (65536 - T). Whole samples take the low half of word 0 of counter
(b, site + 2^31, ...). Seed and offset are an input, two int64 on the GPU.

Tensors are [B, C, H, W] in planar or channels-last memory order.
"""
import functools

import torch

own = False

F32, BF16 = "f32", "bf16"
_DT = {F32: torch.float32, BF16: torch.bfloat16}
_BYTES = {F32: 4, BF16: 2}
SITE = 7
EPS = 1e-6


def _case(name, op, way, B, C, H, W, h=BF16, y=BF16, h_cl=True, y_cl=True, norm="layer", gate="none", drop="none",
          p=0.0, xs=False):
    """h: type of the norm's input or the block's output; y: type of the norm's output or the residual stream;
    h_cl, y_cl: channels-last memory order of each; xs: a residual scale."""
    return {"name": name, "op": op, "way": way, "B": B, "C": C, "H": H, "W": W, "h": h, "y": y, "h_cl": h_cl,
            "y_cl": y_cl, "norm": norm, "gate": gate, "drop": drop, "p": p, "xs": xs}


def listed():
    return [
        # the mixer's planar output of a first-stage block, normalised into the MLP's rows
        _case("norm fwd 56x56 planar-rows", "norm", "fwd", 64, 96, 56, 56, h_cl=False),
        # the same step's gradient in a second-stage block: dy rows from the MLP, dx planar for the mixer
        _case("norm bwd 28x28 planar-rows", "norm", "bwd", 64, 192, 28, 28, h_cl=False),
        # one token of a third-stage width: latency
        _case("norm fwd one token rms", "norm", "fwd", 1, 384, 1, 1, norm="rms"),
        # an odd fp32 plane, odd channel count, planar throughout, as in the parity tests
        _case("norm bwd odd planes f32", "norm", "bwd", 5, 97, 13, 11, h=F32, y=F32, h_cl=False, y_cl=False),
        # the end of a third-stage block with a norm after the MLP, a gate per sample and stochastic depth
        _case("residual fwd 14x14", "residual", "fwd", 64, 384, 14, 14, y_cl=False, norm="rms", gate="sample",
              drop="sample", p=0.1),
        # the layer scale and residual of the level sweep's activations: the largest residual
        _case("residual fwd 128x128 layer scale", "residual", "fwd", 32, 128, 128, 128, y_cl=False, norm="none",
              gate="channel"),
        # the whole gradient of a first-stage block's end, dropout and residual scale included
        _case("residual bwd 56x56", "residual", "bwd", 64, 96, 56, 56, y_cl=False, norm="layer", gate="channel",
              drop="element", p=0.1, xs=True),
        # eight single tokens with a gate each, on an fp32 residual stream
        _case("residual fwd 8 tokens", "residual", "fwd", 8, 768, 1, 1, y=F32, norm="rms", gate="sample"),
        # sequences of tokens in training: fp32 stream, bf16 block, a gate per sample, dropout
        _case("residual bwd 4x2047 tokens", "residual", "bwd", 4, 1024, 1, 2047, y=F32, norm="rms", gate="sample",
              drop="element", p=0.2),
        # the MLP's hidden activations of a first-stage block (4 C channels): the largest of all
        _case("dropout 56x56 hidden rows", "dropout", "fwd", 64, 384, 56, 56, drop="element", p=0.1),
        # odd planar fp32 activations
        _case("dropout odd planes f32", "dropout", "fwd", 3, 97, 57, 55, h=F32, y=F32, h_cl=False, y_cl=False,
              drop="element", p=0.5),
        # one hidden token
        _case("dropout one token", "dropout", "fwd", 1, 1536, 1, 1, drop="element", p=0.1),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["norm", "residual", "residual", "dropout"])
    C = log_int(1, 1536)
    if rng.random() < 0.3:   # tokens: one column of them
        H, W = 1, log_int(1, 4096)
    else:
        H = log_int(1, 128)
        W = max(1, min(128, H + rng.randint(-3, 3)))
    # below the largest listed case: 24 M elements against its 77 M, with fp32 and more tensors a pass
    B = log_int(1, max(1, min(64, 24_000_000 // (C * H * W))))
    h, y = rng.choice([(BF16, BF16), (BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
    h_cl, y_cl = rng.choice([(False, True), (True, False), (True, True), (False, False)])
    way = rng.choice(["fwd", "bwd"])
    norm = rng.choice(["layer", "rms"])
    c = dict(op=op, way=way, B=B, C=C, H=H, W=W, h=h, y=y, h_cl=h_cl, y_cl=y_cl, norm=norm)
    if op == "residual":
        c["norm"] = rng.choice(["none", "layer", "rms"])
        c["gate"] = rng.choice(["none", "channel", "sample"])
        c["drop"] = rng.choice(["none", "element", "sample"])
        c["xs"] = rng.random() < 0.5
    elif op == "dropout":
        c.update(way="fwd", y=h, y_cl=h_cl, drop=rng.choice(["element", "element", "sample"]))
    if c.get("drop", "none") != "none":
        c["p"] = round(rng.uniform(0.02, 0.6), 3)
    c = _case("", **c)
    del c["name"]
    return c


def _layout(t, cl):
    return t.contiguous(memory_format=torch.channels_last) if cl else t.contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    B, C, H, W = case["B"], case["C"], case["H"], case["W"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # activations as they come out of a mixer or an MLP: every channel has a level and a width of its own
    def act(dtype, cl):
        level, width = 0.5 * randn(1, C, 1, 1), torch.exp(0.5 * randn(1, C, 1, 1))
        return _layout((randn(B, C, H, W) * width + level).to(_DT[dtype]), cl)

    s = {"case": case, "h": act(case["h"], case["h_cl"])}
    s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device=dev, dtype=torch.int64)
    s["x"] = s["dy"] = s["weight"] = s["bias"] = s["gate"] = s["xs"] = None
    if case["op"] == "dropout":
        return s
    if case["norm"] != "none":
        s["weight"], s["bias"] = 1 + 0.2 * randn(C), 0.2 * randn(C)
    if case["gate"] != "none":
        s["gate"] = 0.5 * randn(C) if case["gate"] == "channel" else 0.5 * randn(B, C)
    if case["xs"]:
        s["xs"] = 0.5 + torch.rand(C, generator=g, device=dev)
    if case["way"] == "bwd":
        s["dy"] = _layout(randn(B, C, H, W).to(_DT[case["y"]]), case["y_cl"])
    if case["op"] == "residual" and (case["way"] == "fwd" or case["xs"]):
        s["x"] = act(case["y"], case["y_cl"])
    return s


# ---------------------------------------------------------------- plain forms

def _round(state, _):
    c0, c1, c2, c3, k0, k1 = state
    low = 0xFFFFFFFF
    a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57   # 64-bit products, modulo 2^64
    return (((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low,
            (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low)


def _philox(group, site, rng):
    """The four 32-bit words of each counter (group, site, offset), as int64."""
    low = 0xFFFFFFFF
    zero = torch.zeros_like(group)
    start = (group, zero + site, zero + (rng[1] & low), zero + ((rng[1] >> 32) & low), rng[0] & low,
             (rng[0] >> 32) & low)
    return functools.reduce(_round, range(10), start)[:4]


def _keep(case, rng):
    """(keep, scale): the kept elements as a [B, C, H, W] view (samples: [B, 1, 1, 1])."""
    B, C, H, W = case["B"], case["C"], case["H"], case["W"]
    T = int(case["p"] * 65536 + 0.5)
    scale = 65536.0 / (65536 - T) if T < 65536 else 0.0
    if case["drop"] == "sample":
        word = _philox(torch.arange(B, device=rng.device), SITE + (1 << 31), rng)[0]
        return ((word & 0xFFFF) >= T).view(B, 1, 1, 1), scale
    G = -(-C // 8)
    words = torch.stack(_philox(torch.arange(B * H * W * G, device=rng.device), SITE, rng), -1)
    bits = torch.stack((words & 0xFFFF, words >> 16), -1).view(B, H, W, G * 8)[..., :C]
    return (bits >= T).permute(0, 3, 1, 2), scale


def _col(v):
    return v.view(-1, v.shape[-1], 1, 1)


def _normed(case, h):
    """(z, r): the normalised input and the reciprocal deviation of each row."""
    if case["norm"] == "none":
        return h, None
    if case["norm"] == "layer":
        h = h - h.mean(1, keepdim=True)
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    return h * r, r


def _plain(s):
    case = s["case"]
    h = s["h"].float()
    like = {"dtype": _DT[case["y"]], "memory_format": torch.channels_last if case["y_cl"] else torch.contiguous_format}
    if case["op"] == "dropout":
        keep, k = _keep(case, s["rng"])
        return torch.where(keep, h * k, 0.0).to(**like)
    z, r = _normed(case, h)
    v = z if r is None else z * _col(s["weight"]) + _col(s["bias"])
    if case["drop"] != "none":
        keep, k = _keep(case, s["rng"])
    t = v if case["drop"] == "none" else torch.where(keep, v * k, 0.0)
    if case["way"] == "fwd":
        if s["gate"] is not None:
            t = t * _col(s["gate"])
        if s["x"] is not None:
            t = t + (s["x"].float() if s["xs"] is None else s["x"].float() * _col(s["xs"]))
        return t.to(**like)
    dy = s["dy"].float()
    out = {}
    if s["xs"] is not None:
        out["dx"] = (dy * _col(s["xs"])).to(**like)
        out["dxs"] = (dy * s["x"].float()).sum((0, 2, 3))
    if s["gate"] is not None:
        out["dgate"] = (dy * t).sum((0, 2, 3) if case["gate"] == "channel" else (2, 3))
    dv = dy if s["gate"] is None else dy * _col(s["gate"])
    if case["drop"] != "none":
        dv = torch.where(keep, dv * k, 0.0)
    if r is not None:
        out["dweight"], out["dbias"] = (dv * z).sum((0, 2, 3)), dv.sum((0, 2, 3))
        u = dv * _col(s["weight"])
        dv = u - z * (u * z).mean(1, keepdim=True)
        if case["norm"] == "layer":
            dv = dv - u.mean(1, keepdim=True)
        dv = dv * r
    out["dh"] = dv.to(dtype=_DT[case["h"]],
                      memory_format=torch.channels_last if case["h_cl"] else torch.contiguous_format)
    return out


# ------------------------------------------------------- through the library

def _own(s):
    import wavelet_convolution_amd as wt
    case = s["case"]
    if case["op"] == "dropout":
        return wt.wtconv_dropout(s["h"], case["p"], s["rng"], site=SITE, mode=case["drop"])
    if case["op"] == "norm":
        if case["way"] == "fwd":
            return wt.wtconv_norm_fwd(s["h"], s["weight"], s["bias"], kind=case["norm"], eps=EPS,
                                      channels_last=case["y_cl"], dtype=_DT[case["y"]])
        dx, dweight, dbias = wt.wtconv_norm_bwd(s["h"], s["dy"], s["weight"], s["bias"], kind=case["norm"], eps=EPS)
        return {"dweight": dweight, "dbias": dbias, "dh": dx}
    opts = dict(kind=case["norm"], weight=s["weight"], bias=s["bias"], eps=EPS, gate=s["gate"], x_scale=s["xs"],
                drop=case["drop"], p=case["p"], rng=s["rng"], site=SITE)
    if case["way"] == "fwd":
        return wt.wtconv_residual_fwd(s["x"], s["h"], **opts)
    dx, dh, grads = wt.wtconv_residual_bwd(s["dy"], s["h"], x=s["x"], **opts)
    out = {"dh": dh}
    if s["xs"] is not None:
        out.update(dx=dx, dxs=grads[3])
    out.update((n, g) for n, g in zip(("dweight", "dbias", "dgate"), grads) if g is not None)
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    N, eh, ey = case["B"] * case["C"] * case["H"] * case["W"], _BYTES[case["h"]], _BYTES[case["y"]]
    flops = 0
    if case["op"] == "dropout":
        return {"bytes": 2 * N * eh, "flops": 2 * N}
    params = (2 * (case["norm"] != "none") + (case["gate"] == "channel") + case["xs"]) * case["C"] \
        + (case["gate"] == "sample") * case["B"] * case["C"]
    if case["way"] == "fwd":
        tensors = eh + ey + (ey if case["op"] == "residual" else 0)
        flops += N * (2 + 7 * (case["norm"] != "none"))
        return {"bytes": N * tensors + 4 * params, "flops": flops}
    tensors = 2 * eh + ey + (2 * ey if case["xs"] else 0)
    if case["op"] == "residual" and case["norm"] == "none" and case["gate"] == "none":
        tensors -= eh   # nothing that the gradients need is in h
    flops += N * (4 + 16 * (case["norm"] != "none"))
    return {"bytes": N * tensors + 8 * params, "flops": flops}


# ----------------------------------------------- the definition in 64 bits

def _mul32(a, b):
    """(high, low) words of the product of 32-bit a and constant b, from 16-bit halves."""
    a0, a1, b0, b1 = a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16
    mid = a1 * b0 + ((a0 * b0) >> 16)
    mid2 = a0 * b1 + (mid & 0xFFFF)
    return a1 * b1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((a0 * b0) & 0xFFFF)


def _kept_exact(case, rng):
    B, C, H, W = case["B"], case["C"], case["H"], case["W"]
    T = int(case["p"] * 65536 + 0.5)
    seed, off = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    whole = case["drop"] == "sample"
    G = 1 if whole else (C + 7) // 8
    n = torch.arange(B if whole else B * H * W * G, device=rng.device)
    ctr = [n, torch.full_like(n, SITE + (2 ** 31 if whole else 0)), torch.full_like(n, off % 2 ** 32),
           torch.full_like(n, off >> 32)]
    for i in range(10):
        k0 = (seed % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32
        k1 = ((seed >> 32) + i * 0xBB67AE85) % 2 ** 32
        h0, l0 = _mul32(ctr[0], 0xD2511F53)
        h1, l1 = _mul32(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ k0, l1, h0 ^ ctr[3] ^ k1, l0]
    if whole:
        keep = (ctr[0] % 65536 >= T).double().reshape(B, 1, 1, 1)
    else:
        keep = torch.zeros(B * H * W, G * 8, dtype=torch.float64, device=rng.device)
        for j in range(8):
            half = ctr[j // 2] // 65536 if j % 2 else ctr[j // 2] % 65536
            keep[:, j::8] = (half >= T).double().reshape(B * H * W, G)
        keep = keep[:, :C].reshape(B, H, W, C).permute(0, 3, 1, 2)
    return keep * (65536.0 / (65536 - T) if T < 65536 else 0.0)


def exact(case, seed):
    """The operators' definition in 64 bits, their gradients by automatic differentiation of it."""
    s = prepare(case, seed)
    back = case["way"] == "bwd"
    v = {n: s[n].double().requires_grad_(back) for n in ("h", "x", "weight", "bias", "gate", "xs") if s[n] is not None}
    with torch.set_grad_enabled(back):
        t = v["h"]
        if case["op"] != "dropout" and case["norm"] != "none":
            var, mean = torch.var_mean(t, 1, correction=0, keepdim=True)
            if case["norm"] == "layer":
                t = (t - mean) / (var + EPS) ** 0.5
            else:
                t = t / (var + mean ** 2 + EPS) ** 0.5
            t = t * v["weight"][None, :, None, None] + v["bias"][None, :, None, None]
        if case["drop"] != "none":
            t = t * _kept_exact(case, s["rng"])
        if "gate" in v:
            t = t * (v["gate"][:, :, None, None] if case["gate"] == "sample" else v["gate"][None, :, None, None])
        if "x" in v:
            t = t + (v["x"] * v["xs"][None, :, None, None] if "xs" in v else v["x"])
    if not back:
        return t
    names = list(v)
    grads = dict(zip(names, torch.autograd.grad(t, [v[n] for n in names], s["dy"].double())))
    return {"d" + n: g for n, g in grads.items() if n != "x" or "xs" in v}
