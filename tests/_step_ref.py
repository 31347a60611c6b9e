"""Plain 64-bit forms of the expert rows and of the optimizer's step, and the
bounds that fp32 arithmetic allows. U is half a step of fp32 relative to the
value, H that of a type."""
import numpy as np
import torch

from tests._block_ref import philox

U = 2.0 ** -24
BLOCK = 256


def half(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def sort_ref(expert: torch.Tensor, E: int):
    """(order, place, offsets) by numpy's stable sort."""
    e = expert.cpu().numpy().reshape(-1).astype(np.int64)
    key = np.where((e < 0) | (e >= E), E, e)
    order = np.argsort(key, kind="stable")
    place = np.empty_like(order)
    place[order] = np.arange(len(e))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1))[:E]])
    return order, place.reshape(tuple(expert.shape)), offsets


def live_of(place, offsets):
    slots = place.reshape(-1).long()
    return (slots >= 0) & (slots < len(slots)) & (slots < int(offsets[-1]))


def picked(rows, place, offsets):
    """[N, K, C] in 64 bits: each slot's row, zeros without an expert."""
    slots, live = place.reshape(-1).long(), live_of(place, offsets)
    out = torch.zeros(len(slots), rows.shape[-1], dtype=torch.float64, device=rows.device)
    out[live] = rows.double()[slots[live]]
    return out.view(-1, place.shape[-1], rows.shape[-1])


def rows_ref(x, place, offsets):
    """(xs, written): what no place names is not written."""
    slots, live, C = place.reshape(-1).long(), live_of(place, offsets), x.shape[-1]
    each = x.reshape(-1, 1, C).expand(-1, place.shape[-1], C).reshape(-1, C)
    xs, there = torch.zeros_like(each), (slots >= 0) & (slots < len(slots))
    written = torch.zeros(len(slots), dtype=torch.bool, device=x.device)
    xs[slots[live]] = each[live]
    written[slots[there]] = True
    return xs, written


def sum_ref(ys, weight, place, offsets):
    """(y, bound) of the weighted sum; weight None: of ones."""
    q = picked(ys, place, offsets)
    live = live_of(place, offsets).view(q.shape[:2])
    w = live.double() if weight is None else torch.where(live, weight.reshape(live.shape).double(), 0.0)
    terms = w.unsqueeze(-1) * q
    y = terms.sum(1)
    # K fused steps in fp32, each rounded, and the store
    bound = place.shape[-1] * U * 1.01 * terms.abs().sum(1) + half(ys.dtype) * 1.01 * y.abs() + 1e-38
    return y, bound


def sum_bwd_ref(dy, ys, weight, place, offsets):
    """((dys, bound), (dweight, bound)), dys with zeros where no live slot is."""
    C, K = dy.shape[-1], place.shape[-1]
    slots, live = place.reshape(-1).long(), live_of(place, offsets)
    each = dy.reshape(-1, 1, C).double().expand(-1, K, C)
    dys = torch.zeros(len(slots), C, dtype=torch.float64, device=dy.device)
    dys[slots[live]] = (weight.reshape(-1, K, 1).double() * each).reshape(-1, C)[live]
    products = each * picked(ys, place, offsets)
    dweight = products.sum(-1)
    # one product, rounded and stored; a sum of C products in any order
    return ((dys, (U + half(dy.dtype)) * 1.01 * dys.abs() + 1e-38),
            (dweight.view(place.shape), ((C + 8) * U * products.abs().sum(-1) + 1e-38).view(place.shape)))


# ------------------------------------------------------------------ AdamW

def places(params):
    at = 0
    for p in params:
        yield slice(at, at + p.numel())
        at += -(-p.numel() // BLOCK) * BLOCK


def e4m3_steps(q):
    """Distance of e4m3 numbers at q."""
    e = torch.frexp(q.abs().clamp(max=448.0))[1] - 1
    return torch.exp2(e.clamp(min=-6).double() - 3)


def random_bits(count, tensor, site, rng):
    """[count, 2] of the 16 bits for m and v of a tensor's elements."""
    seed, offset = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    words = philox(np.arange(-(-count // 4)), site + tensor, offset, seed).reshape(-1)[:count].astype(np.int64)
    return torch.from_numpy(np.stack([words & 0xFFFF, words >> 16], -1)).double()


def check_codes(what, got, value, err, units, u):
    """Held values `got` (in units) of `value` (64 bits, off by err at most in the kernel): the nearest e4m3 numbers,
    or the ones that the bits u choose, wherever the error does not cross a border."""
    live = units > 0
    unit = torch.where(live, units, 1.0)
    q = torch.where(live, value / unit, 0.0)
    a, step = q.abs().clamp(max=448.0), e4m3_steps(q)
    # the unit and the quotient are rounded too; and the last bit of 2^-20 steps of the random form
    slack = (err / unit + 6 * U * a) / step * 1.01 + 2.0 ** -19
    n = a / step + (0.5 if u is None else (u + 0.5) / 65536)
    want = torch.floor(n)
    if u is None:   # ties go to the even number
        want = torch.where(n == want, torch.round(a / step), want)
    want = torch.copysign(want * step, q)
    border = (n - torch.round(n)).abs() <= slack
    bad = (got != want) & ~border
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], q[bad][:4])
    # at a border one of the two neighbours
    near = (got - want).abs() <= step * 1.01
    assert near[border].all(), (what, "border", got[border & ~near][:4], want[border & ~near][:4])


class Step:
    """One AdamW step on copies of a call's tensors, in 64 bits, and the check of what the call left."""

    def __init__(self, params, grads, m, v, step, *, lr, weight_decay, betas=(0.9, 0.999), eps=1e-8, scales=None,
                 master=None, factor=None, lr_factor=None, rng=None, site=0):
        n = len(params)
        self.lr = [lr] * n if isinstance(lr, float) else [float(x) for x in lr]
        self.wd = [weight_decay] * n if isinstance(weight_decay, float) else [float(x) for x in weight_decay]
        # the host's numbers reach the kernel in fp32
        self.lr, self.wd = (torch.tensor(x, dtype=torch.float32).double().tolist() for x in (self.lr, self.wd))
        self.lr = [x * (1.0 if lr_factor is None else float(lr_factor)) for x in self.lr]
        self.betas, self.eps = betas, eps
        self.f = 1.0 if factor is None else float(factor)
        self.t = max(1, int(step))
        self.rng, self.site = rng, site
        self.params, self.grads = params, grads
        self.now = dict(m=m, v=v, scales=scales, master=master)
        self.old = {k: None if t is None else t.clone() for k, t in self.now.items()}
        self.old_params = [p.clone() for p in params]

    def check(self):
        (b1, b2), eight = self.betas, self.now["scales"] is not None
        c1, c2 = 1 - b1 ** self.t, 1 - b2 ** self.t
        covered = torch.zeros_like(self.old["m"], dtype=torch.bool)
        for i, (p, g, at) in enumerate(zip(self.params, self.grads, places(self.params))):
            what = (i, tuple(p.shape))
            blocks = slice(at.start // BLOCK, -(-at.stop // BLOCK))
            if g is None:
                assert torch.equal(p, self.old_params[i]), what
                continue
            if p.numel() == 0:
                continue
            whole = slice(blocks.start * BLOCK, blocks.stop * BLOCK)
            covered[whole if eight else at] = True
            g = g.detach().reshape(-1).double() * self.f
            m0, v0 = self.old["m"][at].double(), self.old["v"][at].double()
            more = 0.0   # widened states are rounded products of their own
            if eight:
                unit = self.old["scales"][blocks].double().repeat_interleave(BLOCK, 0)[:len(g)]
                m0, v0, more = m0 * unit[:, 0], (v0 * unit[:, 1]) ** 2, 1.0
            m, v = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
            # m: two constants, two products (one more widened), one sum; v likewise with a square
            em = U * 1.01 * ((1 + more) * (b1 * m0).abs() + 3 * ((1 - b1) * g).abs() + m.abs()) + 1e-44
            ev = U * 1.01 * ((1 + 3 * more) * (b2 * v0) + 6 * (1 - b2) * g * g + v) + 1e-44
            root, den = v.sqrt(), (v / c2).sqrt() + self.eps
            # the root to one step of its own; where v is (near) zero, by the square root of v's error
            eroot = torch.minimum(ev / root.clamp(min=1e-300), (2 * ev).sqrt()) + 2 * U * 1.01 * root
            rate = self.lr[i] / c1
            old = (self.old["master"][at] if self.now["master"] is not None
                   else self.old_params[i].reshape(-1)).double()
            update = rate * m / den
            want = old * (1 - self.lr[i] * self.wd[i]) - update
            # in half steps: 1 - b^t 5 (the logarithm and its product with t 2 at most, as |x e^x| < 1 - e^x for x < 0;
            # the series or the power 3); its reciprocal root 4.5; the rate 12 (its factor, that root twice, two
            # products); the denominator 5.5, its reciprocal 2, two products: 21.5 of the update
            ep = U * 1.01 * (4 * old.abs() + 24 * update.abs() + want.abs()) + rate * em / den \
                + update.abs() * (eroot / c2 ** 0.5 / den) + 1e-44
            left = self.now["master"][at] if self.now["master"] is not None else p.detach().reshape(-1)
            bound = ep + (half(p.dtype) * 1.01 * want.abs() if left.dtype == torch.bfloat16 else 0)
            self._near(what + ("p",), left, want, bound)
            if self.now["master"] is not None:
                assert torch.equal(p.detach().reshape(-1), left.to(p.dtype)), what
            if not eight:
                self._near(what + ("m",), self.now["m"][at], m, em)
                self._near(what + ("v",), self.now["v"][at], v, ev)
            else:
                self._check8(what, i, at, blocks, m, em, root, eroot)
        for k in ("m", "v", "master"):
            t = self.now[k]
            if t is not None:
                c = covered if k != "master" else torch.zeros_like(covered)
                if k == "master":
                    for p, g, at in zip(self.params, self.grads, places(self.params)):
                        c[at] = g is not None
                a, b = t.view(torch.uint8 if t.dtype != torch.float32 else torch.int32), \
                    self.old[k].view(torch.uint8 if t.dtype != torch.float32 else torch.int32)
                assert torch.equal(a[~c], b[~c]), k

    @staticmethod
    def _near(what, got, want, bound):
        off = (got.double() - want).abs()
        assert torch.isfinite(got.double()).all(), what
        bad = off > bound
        assert not bad.any(), (what, int(bad.sum()), float((off / bound).max()), got[bad][:3], want[bad][:3])

    def _check8(self, what, i, at, blocks, m, em, root, eroot):
        n = len(m)
        u = None if self.rng is None else random_bits(n, i, self.site, self.rng).to(m.device)
        for k, (name, value, err) in enumerate((("m", m, em), ("v", root, eroot))):
            pad = torch.zeros((blocks.stop - blocks.start) * BLOCK, dtype=torch.float64, device=m.device)
            pad[:n] = value.abs()
            top = pad.view(-1, BLOCK).amax(1)
            pad[:n] = err
            scale, most = self.now["scales"][blocks, k].double(), pad.view(-1, BLOCK).amax(1)
            if name == "m":
                top = torch.where(top < 2.0 ** -100, 0.0, top)
            # the largest of the block and its product with 1 / 448, itself rounded
            off = (scale - top / 448).abs() - (most + 3 * U * top) / 448
            assert (off <= 1e-44).all(), what + (name, "scale", float(off.max()))
            units = scale.repeat_interleave(BLOCK)[:n]
            got = self.now[name][at].double()
            if name == "v":   # a root that is not zero is held as 2^-9 units at least
                value = torch.where(root > 0, torch.maximum(root, units * 2.0 ** -9), root)
                assert (got[root > 1e-37] > 0).all()
            check_codes(what + (name,), got, value, err, units, None if u is None else u[:, k])
            tail = self.now[name][at.stop:blocks.stop * BLOCK].double()
            assert (tail == 0).all() or torch.equal(
                self.now[name][at.stop:blocks.stop * BLOCK].view(torch.uint8),
                self.old[name][at.stop:blocks.stop * BLOCK].view(torch.uint8)), what
