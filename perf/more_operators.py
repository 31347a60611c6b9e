"""The operators of a block's training step that are measured beside the block
operators: rows sorted by expert and back, the gradients' norm and AdamW, in
plain torch operations and through the library.

A block whose MLP is a set of experts sends each of its N rows (pixels or
tokens of C channels) to K of E experts:

    order, place, offsets = sort(expert)         expert [N, K]; slots n * K + k sorted by expert
    xs[place[n, k]] = x[n]                       the experts' rows; slots of no expert (an id outside
    y[n] = sum_k weight[n, k] * ys[place[n, k]]  0..E-1) come last, as rows of zeros, and count nothing

The sort keeps the order of the slots within an expert; expert e's rows are
offsets[e] .. offsets[e + 1] - 1. Backwards

    dx[n] = sum_k dxs[place[n, k]],  dys[place[n, k]] = weight[n, k] * dy[n],
    dweight[n, k] = <dy[n], ys[place[n, k]]>.

The step that follows works on all parameters at once: the norm of all
gradients with the factor min(1, max_norm / (norm + 1e-6)), and AdamW

    g' = factor * g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
    p  = p - lr * wd * p - lr * (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)

with lr and wd per tensor and the step's number t on the GPU. The states of
all tensors stand in one buffer, each tensor's from a multiple of 256 elements
on. In 8 bits a block of 256 elements holds m and sqrt(v) as e4m3 numbers in
units of scales[block] = {max |m|, max sqrt(v)} / 448; a root that is not zero
is held as 2^-9 units at least. They are rounded to the nearest value, or, with
rng (two int64 {seed, offset} on the GPU), up with the probability that makes
the mean right: |q| becomes floor(|q| / step + (u + 1/2) / 65536) * step, u the
low (m) or high (v) 16 bits of word e % 4 of Philox4x32-10 (Salmon, Moraes,
Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with counter
(e // 4, site + tensor, offset low, offset high) and key (seed low, seed high)
for element e of its tensor. bf16 parameters may have an fp32 master copy, laid
out as the states, which is then what the step works on.
"""
import functools

import torch

own = False

F32, BF16 = "f32", "bf16"
_DT = {F32: torch.float32, BF16: torch.bfloat16}
_BYTES = {F32: 4, BF16: 2}
BLOCK = 256
SITE = 100
BETAS = (0.9, 0.999)
EPS = 1e-8
MAX_NORM = 1.0


def _rows(name, op, way, N, C, K, E, t=BF16, dropped=0.0):
    """N rows of C channels to K of E experts; dropped: the share of slots that go to no expert."""
    return {"name": name, "op": op, "way": way, "N": N, "C": C, "K": K, "E": E, "t": t, "dropped": dropped}


def _step(name, op, C, depths, experts=0, p=F32, g=F32, master=False, bits=32, stochastic=False, lr=1e-3, t=100):
    """The tensors of a network of blocks: stages of `depths` blocks, C channels in the first and twice as many in
    each later one, MLPs of `experts` experts (0: one plain MLP)."""
    return {"name": name, "op": op, "C": C, "depths": depths, "experts": experts, "p": p, "g": g, "master": master,
            "bits": bits, "stochastic": stochastic, "lr": lr, "t": t}


def listed():
    return [
        # one token's two experts: latency
        _rows("sort one token", "sort", "fwd", 1, 384, 2, 8),
        # every pixel of a first-stage batch
        _rows("sort 56x56", "sort", "fwd", 64 * 56 * 56, 96, 2, 16),
        # a second-stage block's normalised rows, sent to their experts
        _rows("rows fwd 28x28", "rows", "fwd", 64 * 28 * 28, 192, 2, 16),
        # the gradient of sequences of tokens, some of them padding that goes nowhere, odd length, fp32
        _rows("rows bwd 4x2047 tokens f32", "rows", "bwd", 4 * 2047, 1024, 2, 64, t=F32, dropped=0.1),
        # the experts' results of a first-stage batch, weighted and summed
        _rows("sum fwd 56x56", "sum", "fwd", 64 * 56 * 56, 96, 2, 16),
        # the same sum's gradient in a third-stage block
        _rows("sum bwd 14x14", "sum", "bwd", 64 * 14 * 14, 384, 2, 16),
        # the gradients of a three-stage network in bf16
        _step("norm three stages", "norm", 96, "3,3,27", p=BF16, g=BF16),
        # those of one first-stage block in fp32: latency
        _step("norm one block f32", "norm", 96, "1"),
        # one first-stage block's tensors, small ones most of them: latency
        _step("adamw one block f32", "adamw", 96, "1"),
        # a three-stage network trained in bf16 with fp32 master copies
        _step("adamw three stages master", "adamw", 96, "3,3,27", p=BF16, g=BF16, master=True, lr=5e-4),
        # a block of an odd width whose states are rounded stochastically
        _step("adamw8 odd block f32", "adamw", 97, "2", bits=8, stochastic=True, lr=1e-4),
        # third-stage blocks with 16 experts each, where the states' size counts: the largest
        _step("adamw8 four expert blocks", "adamw", 384, "4", experts=16, p=BF16, g=BF16, master=True, bits=8, lr=5e-5),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["sort", "rows", "sum", "sum", "norm", "adamw", "adamw", "adamw"])
    if op in ("sort", "rows", "sum"):
        E = log_int(1, 256)
        K = min(E, rng.choice([1, 2, 2, 3, 4, 8]))
        C = log_int(1, 1536)
        # below the largest listed case: 24 M elements
        N = log_int(1, max(1, min(200_704, 24_000_000 // (C * K))))
        way = "fwd" if op == "sort" else rng.choice(["fwd", "bwd"])
        c = _rows("", op, way, N, C, K, E, t=rng.choice([F32, BF16]), dropped=rng.choice([0.0, 0.0, 0.05, 0.5]))
    else:
        while True:
            C, experts = log_int(8, 384), rng.choice([0, 0, 0, 2, 4, 8])
            depths = [rng.randint(1, 4) for _ in range(rng.randint(1, 4))]
            if sum(n * 8 * (C << s) ** 2 * max(1, experts) for s, n in enumerate(depths)) < 30_000_000:
                break
        p, g, master = rng.choice([(F32, F32, False), (F32, BF16, False), (BF16, BF16, True), (BF16, F32, True),
                                   (BF16, BF16, False)])
        bits = 32 if op == "norm" else rng.choice([8, 32])
        # up to a training run's rate; with states in 8 bits up to fine-tuning's
        lr = round(10.0 ** rng.uniform(-5, -4 if bits == 8 else -2.5), 7)
        c = _step("", op, C, ",".join(map(str, depths)), experts, p, g, master, bits,
                  bits == 8 and rng.random() < 0.5, lr, log_int(1, 100_000))
    del c["name"]
    return c


def _shapes(case):
    """The parameters of the case's blocks: base and level kernels, scales, norm, MLP (or experts), layer scale."""
    out = []
    for s, depth in enumerate(map(int, case["depths"].split(","))):
        C, L, E = case["C"] << s, max(1, 3 - s), case["experts"]
        mlp = [(4 * C, C), (4 * C,), (C, 4 * C), (C,)]
        block = [(C, 5, 5), (L, C, 4, 5, 5), (L, C, 4), (C,), (C,), *([(E, *m) for m in mlp] if E else mlp), (C,)]
        out += block * depth
    return out


def _count(shape):
    return functools.reduce(lambda a, b: a * b, shape, 1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": case}
    if case["op"] in ("sort", "rows", "sum"):
        N, C, K, E, t = case["N"], case["C"], case["K"], case["E"], _DT[case["t"]]
        # a router that likes some experts better than others
        logits = randn(N, E) + 0.7 * randn(E)
        top, expert = logits.topk(K, 1)
        expert = torch.where(torch.rand(N, K, generator=g, device=dev) < case["dropped"], -1, expert)
        s["expert"] = expert
        if case["op"] != "sort":
            s["order"], s["place"], s["offsets"] = _sort(expert, E)
            s["weight"] = torch.softmax(top, 1)
            if (case["op"], case["way"]) in (("rows", "fwd"), ("sum", "bwd")):
                s["rows"] = randn(N, C).to(t)
            if (case["op"], case["way"]) != ("rows", "fwd"):
                s["sorted"] = randn(N * K, C).to(t)
        return s
    shapes = _shapes(case)
    blocks = [-(-_count(x) // BLOCK) for x in shapes]
    n, start = sum(blocks) * BLOCK, [0]
    for b in blocks:
        start.append(start[-1] + b * BLOCK)

    def views(flat):
        return [flat[a:a + _count(x)].view(x) for a, x in zip(start, shapes)]

    # gradients and parameters as views of one buffer each, zero between the tensors; every tensor has a width of
    # its own, and a gradient's elements have widths that differ as the moments' do
    s["blocks"] = torch.tensor(blocks, device=dev)
    used = torch.zeros(n, device=dev)
    for u in views(used):
        u.fill_(1)
    width = torch.repeat_interleave(torch.exp(0.5 * randn(len(shapes))), s["blocks"]).repeat_interleave(BLOCK) * used
    wide = 1e-3 * width * torch.exp(randn(n))
    s["grad"] = (wide * randn(n)).to(_DT[case["g"]])
    s["grads"] = views(s["grad"])
    if case["op"] == "norm":
        return s
    master = 0.02 * width * randn(n)
    s["param"] = master.to(_DT[case["p"]])
    s["params"] = views(s["param"])
    s["master"] = master if case["master"] else None
    s["step"] = torch.full((1,), case["t"], dtype=torch.int64, device=dev)
    s["factor"] = 0.5 + 0.5 * torch.rand(1, generator=g, device=dev)
    s["lr"] = torch.tensor([case["lr"] * (0.9 ** (i % 3)) for i in range(len(shapes))])
    s["wd"] = torch.tensor([0.05 if len(x) > 1 else 0.0 for x in shapes])
    s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device=dev, dtype=torch.int64) if case["stochastic"] else None
    # the states that earlier steps with such gradients leave
    m, v = 0.3 * wide * randn(n), (wide * (0.7 + 0.6 * torch.rand(n, generator=g, device=dev))) ** 2
    if case["bits"] == 32:
        s["m"], s["v"], s["scales"] = m, v, None
    else:
        s["m"], s["v"], s["scales"] = _to8(m.double(), v.double().sqrt(), None)
    return s


# ---------------------------------------------------------------- plain forms

def _sort(expert, E):
    e = expert.reshape(-1)
    key = torch.where((e < 0) | (e >= E), E, e)
    order = torch.sort(key, stable=True)[1]
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    # the first sorted slot of each expert: how many slots have a smaller one
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=key.device))
    return order.int(), place.int().view(expert.shape), offsets.int()


def _kept(s):
    return (s["place"] < s["offsets"][-1]).unsqueeze(-1)


def _plain_rows(s):
    case, place = s["case"], s["place"].long()
    t, kept = _DT[case["t"]], _kept(s)
    if case["op"] == "rows" and case["way"] == "fwd":
        out = torch.empty(place.numel(), case["C"], dtype=t, device=place.device)
        out[place.view(-1)] = torch.where(kept, s["rows"].unsqueeze(1), 0).view(-1, case["C"])
        return out
    rows = torch.where(kept, s["sorted"][place].float(), 0)
    if case["op"] == "rows":
        return rows.sum(1).to(t)
    if case["way"] == "fwd":
        return (rows * s["weight"].unsqueeze(-1)).sum(1).to(t)
    dy = s["rows"].float().unsqueeze(1)
    dys = torch.empty_like(s["sorted"])
    dys[place.view(-1)] = torch.where(kept, dy * s["weight"].unsqueeze(-1), 0).to(t).view(-1, case["C"])
    return {"dys": dys, "dweight": (rows * dy).sum(-1)}


def _round(state, _):
    c0, c1, c2, c3, k0, k1 = state
    low = 0xFFFFFFFF
    a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57   # 64-bit products, modulo 2^64
    return (((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low,
            (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low)


def _bits(s):
    """[elements, 2] of 16 bits for each element of the states' buffer, as int64."""
    low, rng, blocks = 0xFFFFFFFF, s["rng"], s["blocks"]
    tensor = torch.repeat_interleave(torch.arange(len(blocks), device=rng.device), blocks)
    first = torch.repeat_interleave(torch.cumsum(blocks, 0) - blocks, blocks)
    block = torch.arange(len(tensor), device=rng.device) - first
    group = (block.unsqueeze(1) * (BLOCK // 4) + torch.arange(BLOCK // 4, device=rng.device)).view(-1)
    site = (tensor + SITE).repeat_interleave(BLOCK // 4)
    zero = torch.zeros_like(group)
    start = (group, site, zero + (rng[1] & low), zero + ((rng[1] >> 32) & low), rng[0] & low, (rng[0] >> 32) & low)
    word = torch.stack(functools.reduce(_round, range(10), start)[:4], -1).view(-1)
    return torch.stack((word & 0xFFFF, word >> 16), -1)


def _e4m3(q, u):
    """q (64 bits, |q| <= 448) as e4m3 numbers: the nearest, or up by the 16 bits u."""
    a = q.abs().clamp(max=448.0)
    step = torch.exp2(torch.clamp(torch.frexp(a)[1] - 1, min=-6).double() - 3)
    n = a / step
    return torch.copysign((torch.round(n) if u is None else torch.floor(n + (u + 0.5) / 65536)) * step, q)


def _to8(m, root, u):
    """(m, v, scales) in 8 bits of the first moment and the second one's root, in 64 bits: a value next to the border
    between two of the 8-bit numbers has to fall on its own side."""
    both = torch.stack((m, root)).view(2, -1, BLOCK)
    scale = (both.abs().amax(-1) / 448).float()
    unit = torch.where(scale > 0, scale, 1.0).double().unsqueeze(-1)
    qm, qv = (both / unit).view(2, -1)
    qm, qv = _e4m3(qm, None if u is None else u[:, 0]), _e4m3(qv, None if u is None else u[:, 1])
    qv = torch.where(root > 0, torch.clamp(qv, min=2.0 ** -9), qv)
    return qm.to(torch.float8_e4m3fn), qv.to(torch.float8_e4m3fn), scale.t().contiguous()


def _plain_norm(s):
    norm = s["grad"].double().square().sum().sqrt()
    return torch.stack((norm, torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0))).float()


def _plain_adamw(s):
    case, (b1, b2) = s["case"], BETAS
    t = s["step"].double()
    c1, c2 = (1 - b1 ** t).float(), (1 - b2 ** t).float()
    lr, wd = (torch.repeat_interleave(s[n].to(t.device), s["blocks"]).unsqueeze(1) for n in ("lr", "wd"))
    x = s["param"] if s["master"] is None else s["master"]
    p, g = x.float(), s["grad"].float() * s["factor"]
    if case["bits"] == 32:
        m = s["m"].mul_(b1).add_((1 - b1) * g)
        v = s["v"].mul_(b2).add_((1 - b2) * g * g)
        root = torch.sqrt(v)
    else:
        g = g.double()
        unit = s["scales"].double()
        m = s["m"].double().view(-1, BLOCK) * unit[:, :1]
        root = s["v"].double().view(-1, BLOCK) * unit[:, 1:]
        m = b1 * m.view(-1) + (1 - b1) * g
        root = torch.sqrt(b2 * root.view(-1) ** 2 + (1 - b2) * g * g)
        u = None if s["rng"] is None else _bits(s)
        for old, new in zip((s["m"], s["v"], s["scales"]), _to8(m, root, u)):
            old.copy_(new)
        m, root = m.float(), root.float()
    update = m / c1 / (root / torch.sqrt(c2) + EPS)
    p = (p.view(-1, BLOCK) * (1 - lr * wd) - lr * update.view(-1, BLOCK)).view(-1)
    if s["master"] is not None:
        s["master"].copy_(p)
    s["param"].copy_(p)
    return _outputs(s)


def _outputs(s):
    return {n: s[n] for n in ("param", "master", "m", "v", "scales") if s[n] is not None}


def _plain(s):
    op = s["case"]["op"]
    if op == "sort":
        return _sort(s["expert"], s["case"]["E"])
    return _plain_norm(s) if op == "norm" else _plain_adamw(s) if op == "adamw" else _plain_rows(s)


# ------------------------------------------------------- through the library

def _own(s):
    import wavelet_convolution_amd as wt
    case, op = s["case"], s["case"]["op"]
    if op == "sort":
        return wt.wtconv_expert_sort(s["expert"], case["E"])
    if op == "rows":
        if case["way"] == "fwd":
            return wt.wtconv_expert_rows_fwd(s["rows"], s["place"], s["offsets"])
        return wt.wtconv_expert_rows_bwd(s["sorted"], s["place"], s["offsets"])
    if op == "sum":
        if case["way"] == "fwd":
            return wt.wtconv_expert_sum_fwd(s["sorted"], s["weight"], s["place"], s["offsets"])
        dys, dweight = wt.wtconv_expert_sum_bwd(s["rows"], s["sorted"], s["weight"], s["place"], s["offsets"])
        return {"dys": dys, "dweight": dweight}
    if op == "norm":
        return wt.wtconv_grad_norm(s["grads"], MAX_NORM)
    wt.wtconv_adamw_step(s["params"], s["grads"], s["m"], s["v"], s["step"], scales=s["scales"], master=s["master"],
                         lr=s["lr"], betas=BETAS, eps=EPS, weight_decay=s["wd"], factor=s["factor"], rng=s["rng"],
                         site=SITE)
    return _outputs(s)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    if case["op"] in ("sort", "rows", "sum"):
        S, e = case["N"] * case["K"], _BYTES[case["t"]]
        row, table = case["C"] * e, 4 * S
        if case["op"] == "sort":   # ids of 64 bits in, order and place out
            return {"bytes": 16 * S + 4 * (case["E"] + 1), "flops": 0}
        if case["op"] == "rows":
            return {"bytes": case["N"] * row + S * row + table, "flops": 0 if case["way"] == "fwd" else S * case["C"]}
        if case["way"] == "fwd":
            return {"bytes": case["N"] * row + S * row + 2 * table, "flops": 2 * S * case["C"]}
        return {"bytes": case["N"] * row + 2 * S * row + 3 * table, "flops": 3 * S * case["C"]}
    n, eg = sum(map(_count, _shapes(case))), _BYTES[case["g"]]
    if case["op"] == "norm":
        return {"bytes": n * eg + 8, "flops": 2 * n}
    param = 8 + _BYTES[case["p"]] if case["master"] else 2 * _BYTES[case["p"]]
    states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": int(n * (eg + param + states)), "flops": n * (16 if case["bits"] == 32 else 30)}


# ----------------------------------------------- the definition in 64 bits

def _exact_rows(case, s):
    slots = s["place"].reshape(-1).long()
    live = (slots < int(s["offsets"][-1])).double()
    # row i of the matrix [N, S] of the routing, applied without building it
    back = case["way"] == "bwd"
    if case["op"] == "rows":
        if not back:
            source = torch.div(torch.argsort(slots), case["K"], rounding_mode="floor")
            alive = (torch.arange(len(slots), device=slots.device) < int(s["offsets"][-1])).double()
            return s["rows"].double()[source] * alive[:, None]
        picked = s["sorted"].double()[slots] * live[:, None]
        return torch.stack([picked[k::case["K"]] for k in range(case["K"])]).sum(0)
    ys = s["sorted"].double().requires_grad_(back)
    weight = s["weight"].double().requires_grad_(back)
    with torch.set_grad_enabled(back):
        y = 0
        for k in range(case["K"]):
            y = y + (weight[:, k] * live[k::case["K"]])[:, None] * ys[slots[k::case["K"]]]
    if not back:
        return y
    dys, dweight = torch.autograd.grad(y, (ys, weight), s["rows"].double())
    return {"dys": dys, "dweight": dweight}


def exact(case, seed):
    """The operators' definition in 64 bits. Where a state is held in 8 bits, the value before that rounding, in the
    same units; a sort has whole numbers only."""
    if case["op"] == "sort":
        return None
    s = prepare(case, seed)
    if case["op"] in ("rows", "sum"):
        return _exact_rows(case, s)
    grads = [x.double() for x in s["grads"]]
    if case["op"] == "norm":
        norm = sum(float((x * x).sum()) for x in grads) ** 0.5
        return torch.tensor([norm, min(1.0, MAX_NORM / (norm + 1e-6))], dtype=torch.float64)
    t, f = case["t"], float(s["factor"])
    c1, c2 = (1 - b ** t for b in BETAS)
    whole = s["param"] if s["master"] is None else s["master"]
    p, m, v = (torch.zeros(whole.shape, dtype=torch.float64, device=whole.device) for _ in range(3))
    at = 0
    for i, g in enumerate(grads):
        n = g.numel()
        here, pad = slice(at, at + n), slice(at, at + -(-n // BLOCK) * BLOCK)
        g = g.reshape(-1) * f
        if case["bits"] == 32:
            m0, v0 = s["m"][here].double(), s["v"][here].double()
        else:
            unit = s["scales"][pad.start // BLOCK:pad.stop // BLOCK].double().repeat_interleave(BLOCK, 0)[:n]
            m0, v0 = s["m"][here].double() * unit[:, 0], (s["v"][here].double() * unit[:, 1]) ** 2
        m[here] = BETAS[0] * m0 + (1 - BETAS[0]) * g
        v[here] = BETAS[1] * v0 + (1 - BETAS[1]) * g ** 2
        old, lr, wd = whole[here].double(), float(s["lr"][i]), float(s["wd"][i])
        p[here] = old - lr * (wd * old + m[here] / c1 / ((v[here] / c2) ** 0.5 + EPS))
        at = pad.stop
    out = {"param": p, "m": m, "v": v}
    if s["master"] is not None:
        out["master"] = p
    if case["bits"] == 8:
        both = torch.stack((m.abs(), v.sqrt()), 1).view(-1, BLOCK, 2)
        scales = both.amax(1) / 448
        unit = torch.where(scales > 0, scales, 1).repeat_interleave(BLOCK, 0)
        out.update(scales=scales, m=m / unit[:, 0], v=v.sqrt() / unit[:, 1])
    return out
