"""Parameter gradients of the block operators on data whose sums are exact.

The bounds of tests/_block_ref.py grow with the number of rows and can hide a
lost tile among many. Here every product and every partial sum, in any order
and however it is split, is a multiple of a power of two with fewer than 2^24
steps, so fp32 holds it exactly and the gradients have to be equal to the
64-bit sums:
  dy, and h without a norm: -1, 0, 1; x: -2 .. 2; gates, weights, x_scale:
  powers of two; p = 1/2, so what is kept is doubled.
  With a norm: eps = 1 and h = -2^-13, 0, 2^-13 in neighbouring channels of
  opposite sign. Each wavefront's mean is zero, the variance is at most 2^-26,
  and 1 + 2^-26 rounds to 1 in fp32 (half a step is 2^-24): r = 1, z = h."""
import itertools

import pytest
import torch

from tests._block_ref import keep_mask
from tests.test_block import DT, FULL, GENERIC, ORDERS, PAIRS, ROWS, SHAPES, _order, _shape_id, on_gpu
from wavelet_convolution_amd import block_binding as bb

STEP = 2.0 ** -13
RNG = (0x0FEDCBA987654321, 5 + (7 << 33))
SITE = 11
NAMES = ("dweight", "dbias", "dgate", "dx_scale")
MODES = list(itertools.product(("layer", "none", "rms"), ("channel", "sample"), ("none", "element", "sample")))


def data(shape, kind, gate, seed):
    """Inputs on the CPU, in fp32, planar."""
    g = torch.Generator().manual_seed(seed)
    B, C = shape[:2]

    def ints(most, *size):
        return torch.randint(-most, most + 1, size, generator=g, dtype=torch.int8).float()

    def powers(*size):
        return torch.randint(0, 2, size, generator=g) * 2.0 - 1, 2.0 ** torch.randint(-1, 2, size, generator=g)

    d = dict(dy=ints(1, *shape), x=ints(2, *shape), gate=torch.mul(*powers(*((B, C) if gate == "sample" else (C,)))),
             x_scale=torch.mul(*powers(C)), weight=None, bias=None)
    if kind == "none":
        d["h"] = ints(1, *shape)
    else:
        half = ints(1, B, C // 2, 1, *shape[2:]) * STEP
        d["h"] = torch.cat((half, -half), 2).reshape(B, C // 2 * 2, *shape[2:])
        if C % 2:
            d["h"] = torch.cat((d["h"], torch.zeros(B, 1, *shape[2:])), 1)
        d["weight"], d["bias"] = torch.mul(*powers(C)), ints(2, C) * STEP
    return d


def sums(d, kind, gate, drop, count=None):
    """dweight, dbias, dgate, dx_scale in 64 bits; count [B, 1, H, W]: how often each pixel is taken (once)."""
    f = {n: None if t is None else t.double() for n, t in d.items()}
    dy = f["dy"] if count is None else f["dy"] * count
    mask, k = keep_mask(d["h"].shape, drop, 0.5, *RNG, SITE)

    def col(v):
        return v.view(-1, v.shape[-1], 1, 1)

    rows = (0, 2, 3)
    t = f["h"] if kind == "none" else f["h"] * col(f["weight"]) + col(f["bias"])
    t = t * mask * k
    dv = dy * col(f["gate"]) * mask * k
    terms = dict(dgate=(dy * t, (2, 3) if gate == "sample" else rows), dx_scale=(dy * f["x"], rows))
    if kind != "none":
        terms.update(dweight=(dv * f["h"], rows), dbias=(dv, rows))
    for n, (v, dims) in terms.items():   # steps of half a power's product at least
        assert float(v.abs().sum(dims).max()) < 2 ** 24 * (STEP / 4 if kind != "none" and n in ("dweight", "dgate")
                                                            else 0.5), n
    return {n: v.sum(dims) for n, (v, dims) in terms.items()}


def run_case(shape, h_dt, y_dt, order, kind, gate, drop, seed):
    print(f"[exact] {shape} {order} {kind} {gate} {drop} {h_dt} {y_dt}", flush=True)
    d = data(shape, kind, gate, seed)
    h, x, dy = (_order(d[n].to(DT[dt]), cl).cuda() for n, dt, cl in
                (("h", h_dt, order[0]), ("x", y_dt, order[1]), ("dy", y_dt, order[1])))
    p = {n: None if d[n] is None else d[n].cuda() for n in ("weight", "bias", "gate", "x_scale")}
    rng = torch.tensor(RNG, dtype=torch.int64, device="cuda")
    _, _, grads = bb.wtconv_residual_bwd(dy, h, x=x, kind=kind, eps=1.0, drop=drop, p=0.5, rng=rng, site=SITE, **p)
    torch.cuda.synchronize()
    want = sums(d, kind, gate, drop)
    for n, got in zip(NAMES, grads):
        assert (got is None) == (n not in want)
        if got is not None:
            off = (got.double().cpu() != want[n]).nonzero()
            assert not len(off), (n, len(off), off[0].tolist())
    if kind == "none":
        return
    got = bb.wtconv_norm_bwd(h, dy, p["weight"], p["bias"], kind=kind, eps=1.0)[1:]
    torch.cuda.synchronize()
    d["gate"] = torch.ones(shape[1])
    want = sums(d, kind, "channel", "none")
    for n, t in zip(NAMES, got):
        assert torch.equal(t.double().cpu(), want[n]), f"norm {n}"


@on_gpu
@pytest.mark.parametrize("order", [o for o in ORDERS if o != (1, 1)])
@pytest.mark.parametrize("shape", FULL + GENERIC, ids=_shape_id)
def test_planar_sides(shape, order):
    """Grids that fill the card with eight bf16 pixels a lane, and the generic kernels."""
    n = sum(shape) + 5 * order[0] + 11 * order[1]
    for i in range(4):   # every gate twice, every norm and drop at least once
        kind, gate, drop = MODES[(n + 7 * i) % len(MODES)]
        h_dt, y_dt = ("bf16", "bf16") if shape in FULL else PAIRS[(n + i) % 4]
        run_case(shape, h_dt, y_dt, order, kind, gate, drop, seed=n + i)


@on_gpu
@pytest.mark.parametrize("shape", [(64, 96, 56, 56), (9, 72, 1, 300), (3, 100, 17, 33)], ids=_shape_id)
def test_planar_sides_in_every_mode(shape):
    for i, (kind, gate, drop) in enumerate(MODES):
        if shape[0] < 64 or i % 5 == 2:
            run_case(shape, *PAIRS[i % 4 if shape[0] < 64 else 0], ORDERS[i % 3], kind, gate, drop, seed=i)


@on_gpu
@pytest.mark.parametrize("shape", [*SHAPES, *ROWS, (300, 8, 9, 11), (41, 97, 13, 17), (5000, 33, 1, 1),
                                   (7, 1000, 31, 33), (64, 2056, 1, 9)], ids=_shape_id)
def test_rows(shape):
    n = sum(shape)
    for i in range(4):
        kind, gate, drop = MODES[(n + 7 * i) % len(MODES)]
        run_case(shape, *PAIRS[(n + i) % 4], (1, 1), kind, gate, drop, seed=n + i)


# ------------------------------------------------------------------- CPU

@pytest.mark.parametrize("shape,tile", [((350, 96, 9, 13), 64), ((1030, 30, 9, 13), 128), ((5, 72, 90, 97), 64),
                                        ((2, 3, 600, 500), 256), ((64, 7, 20, 21), 8)], ids=str)
def test_these_sums_show_what_a_bound_hides(shape, tile):
    """A sample's first tile left out, its last pixels counted twice, and one pixel left out: each changes every one
    of the sums (of few channels one of them at least: a few pixels' products of -1, 0 and 1 may add up to nothing)."""
    B, C, H, W = shape
    for kind, gate, drop in (("layer", "channel", "none"), ("rms", "sample", "element")):
        d = data(shape, kind, gate, seed=1)
        want = sums(d, kind, gate, drop)
        for first, last, times in ((0, tile, 0), (H * W - 3, H * W, 2), (H * W - 1, H * W, 0)):
            count = torch.ones(B, H * W)
            count[B // 2, first:last] = times
            other = sums(d, kind, gate, drop, count.view(B, 1, H, W))
            seen = [not torch.equal(want[n], other[n]) for n in NAMES]
            assert all(seen) if C > 7 or last == tile else any(seen), (first, last, times, seen)


def test_the_norm_of_this_data_is_the_data():
    """In fp32 and 64 bits alike the normalised input is the input, of odd and even widths, in either norm."""
    for C in (2, 7, 30, 97, 2049):
        h = data((3, C, 2, 5), "layer", "channel", seed=C)["h"]
        assert torch.equal(h.sum(1), torch.zeros(3, 2, 5)) and float(h.abs().max()) == STEP
        for t in (h, h.double()):
            var = t.square().mean(1, keepdim=True)
            assert float(var.max()) <= STEP ** 2
            if t.dtype == torch.float32:
                assert torch.equal(t * (var + 1.0).rsqrt(), h)
        assert torch.equal(h.to(torch.bfloat16).float(), h)


@on_gpu
@pytest.mark.parametrize("C", [1, 3, 7, 8, 32])
def test_sums_over_many_rows_are_short_chains(C):
    """One dout of 2^24 before many of 1: an fp32 sum of 2^24 and 1 stays at 2^24, so a chain of n additions after
    the large one loses n. Additions that any term passes, at the most: a row of its lane, 32 of the groups of a
    workgroup and 4 that join them; in the second stage one slot a lane, 4 over lanes and 16 wavefronts: 58, each of
    them off by half a step of a number up to 2^24 + n < 2^25, 2^-24 of it: 1.002 for these 19,650 rows."""
    n = 19650
    shape = (1, C, 1, n)
    dy = torch.ones(shape, device="cuda")
    dy[..., 0] = 2.0 ** 24
    one = torch.ones(shape, device="cuda")
    dy, one = _order(dy, 1), _order(one, 1)
    want = 2.0 ** 24 + (n - 1)
    xs = torch.ones(C, device="cuda")
    for gate in (torch.ones(C, device="cuda"), torch.ones(1, C, device="cuda")):
        print(f"[chains] {C} {tuple(gate.shape)}", flush=True)
        _, _, (_, _, dgate, dxs) = bb.wtconv_residual_bwd(dy, one, x=one, gate=gate, x_scale=xs)
        _, _, (_, dbias, _, _) = bb.wtconv_residual_bwd(dy, one, gate=gate, kind="rms", bias=torch.zeros(C, device="cuda"))
        for name, t in (("dgate", dgate), ("dx_scale", dxs), ("dbias", dbias)):
            off = (t.double().cpu() - want).abs().max()
            assert float(off) <= 58 * 1.002, (name, float(off))
