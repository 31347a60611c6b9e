"""The optimizer's step: the gradients' norm and AdamW over many tensors,
against the definition in 64 bits (tests/_step_ref.py)."""
import copy
import math

import pytest
import torch

from tests._step_ref import BLOCK, Step, U, places
from wavelet_convolution_amd import AdamW, block_residual, channel_norm, dropout_rng, expert_rows, expert_sort, expert_sum
from wavelet_convolution_amd import optim_binding as ob

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16

# around a vector of four, a block of 256, a workgroup's 4,096; odd shapes, nothing
SHAPES = [(1,), (0,), (3,), (4, 1), (5,), (255,), (16, 16), (257,), (97, 5, 5), (64, 64), (4097,), (2, 0, 3), (3, 97, 4, 5, 5),
          (1021, 33)]


class Call:
    """A call's tensors, filled from a seed."""

    def __init__(self, shapes=SHAPES, p=F32, g=F32, master=False, bits=32, seed=0, t=7, random=False, fresh=False,
                 unaligned=False, missing=(), factor=0.7, lr_factor=None, width=1e-3, **opts):
        gen = torch.Generator(DEV).manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=gen, device=DEV)

        def place(x):
            if not unaligned:
                return x
            y = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape)
            return y.copy_(x)

        self.params = [place((0.05 * randn(*s)).to(p)) for s in shapes]
        self.grads = [None if i in missing else place((width * torch.exp(randn(*s)) * randn(*s)).to(g))
                      for i, s in enumerate(shapes)]
        n = ob.wtconv_adamw_state_count(self.params)
        m, root = (0.3 * width * randn(n)) * (not fresh), (width * (0.5 + torch.rand(n, generator=gen, device=DEV))) * (not fresh)
        self.scales = None
        if bits == 8:
            both = torch.stack((m, root)).view(2, -1, BLOCK)
            self.scales = (both.abs().amax(-1) / 448).t().contiguous()
            unit = torch.where(self.scales > 0, self.scales, 1.0)
            m, v = ((both[i] / unit[:, i:i + 1]).view(-1).to(torch.float8_e4m3fn) for i in range(2))
        else:
            v = root ** 2
        self.m, self.v, self.master = m, v, None
        if master:
            self.master = 0.05 * randn(n)
            for q, at in zip(self.params, places(self.params)):
                self.master[at] += q.reshape(-1).float()
        self.step = torch.full((1,), t, dtype=torch.int64, device=DEV)
        self.opts = dict(lr=1e-3, weight_decay=0.05, scales=self.scales, master=self.master,
                         factor=None if factor is None else torch.full((1,), factor, device=DEV),
                         lr_factor=None if lr_factor is None else torch.full((1,), lr_factor, device=DEV),
                         rng=torch.tensor([seed + 2 ** 40, seed + 2 ** 33], device=DEV) if random else None, site=5 if random else 0)
        self.opts.update(opts)

    def args(self):
        return self.params, self.grads, self.m, self.v, self.step

    def run(self, **kw):
        ob.wtconv_adamw_step(*self.args(), **self.opts, **kw)

    def check(self, **kw):
        want = Step(*self.args(), **self.opts)
        self.run(**kw)
        torch.cuda.synchronize()
        want.check()

    def tensors(self):
        return [t for t in (*self.params, self.m, self.v, self.scales, self.master) if t is not None]

    def bits(self):
        return [t.clone().view(-1).view(torch.uint8) for t in self.tensors()]


KINDS = [(F32, F32, False), (F32, BF16, False), (BF16, BF16, True), (BF16, F32, True), (BF16, BF16, False), (BF16, F32, False)]
STATES = [(32, False), (8, False), (8, True)]


@pytest.mark.parametrize("bits,random", STATES)
@pytest.mark.parametrize("p,g,master", KINDS)
def test_step(p, g, master, bits, random):
    Call(p=p, g=g, master=master, bits=bits, random=random).check()


@pytest.mark.parametrize("bits,random", STATES)
@pytest.mark.parametrize("p,g,master", KINDS)
def test_step_on_pointers_aligned_to_the_element_only(p, g, master, bits, random):
    Call(p=p, g=g, master=master, bits=bits, random=random, seed=1, unaligned=True).check()


@pytest.mark.parametrize("bits,random", STATES)
@pytest.mark.parametrize("t", [-3, 0, 1, 2, 1000, 10 ** 6, 2 ** 40])
def test_first_and_late_steps(t, bits, random):
    """States of zeros at the first step; a count below 1 is 1."""
    Call(bits=bits, random=random, seed=2, t=t, fresh=t <= 1).check()


@pytest.mark.parametrize("bits,random", STATES)
def test_several_steps(bits, random):
    c = Call(bits=bits, random=random, fresh=True, t=1, seed=3)
    for i in range(6):
        c.check()
        c.step += 1
        if random:
            c.opts["rng"][1] += 1
        for j, g in enumerate(c.grads):
            g.copy_(torch.randn(g.shape, device=DEV) * 1e-3 * (i + 1))


@pytest.mark.parametrize("bits,random", STATES)
def test_more_tensors_than_a_launch_takes(bits, random):
    """200 tensors, rates and decays of their own, some without a gradient (runs of them too)."""
    shapes = [((i * 37) % 600 + 1,) for i in range(200)]
    Call(shapes, bits=bits, random=random, seed=4, missing=(0, 5, 79, 80, 81, *range(150, 180), 199),
         lr=torch.linspace(0, 1e-2, 200), weight_decay=[0.1 * (i % 3) for i in range(200)], lr_factor=0.25).check()


@pytest.mark.parametrize("bits", [32, 8])
def test_rates_of_every_tensor(bits):
    """As many rates as tensors: more than a launch's table holds."""
    n = 50
    Call([(130,)] * n, bits=bits, seed=15, lr=[1e-3 * (1 + i) for i in range(n)], weight_decay=torch.linspace(0, 1, n)).check()


@pytest.mark.parametrize("bits", [32, 8])
def test_large_tensor(bits):
    """Several rounds of workgroups over the card, beside small tensors."""
    Call([(7,), (5_000_011,), (300,)], p=BF16, g=BF16, master=True, bits=bits, random=bits == 8, seed=5).check()


def test_betas_and_eps():
    for betas, eps in (((0.0, 0.0), 1e-8), ((0.0, 0.99), 1e-3), ((0.95, 0.0), 1e-6), ((0.5, 0.9999), 1.0)):
        for bits in (32, 8):
            Call(bits=bits, betas=betas, eps=eps, seed=6, t=3).check()


@pytest.mark.parametrize("bits,random", STATES)
@pytest.mark.parametrize("factor", [float("nan"), float("inf"), -float("inf")])
def test_a_factor_that_is_not_finite_changes_nothing(factor, bits, random):
    c = Call(bits=bits, random=random, factor=factor, seed=7)
    c.grads[3][0] = float("nan")
    before = c.bits()
    c.run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, c.bits()))


@pytest.mark.parametrize("bits,random", STATES)
def test_zero_gradients(bits, random):
    """From zero states nothing but the decay changes a parameter, and states stay zero."""
    c = Call(bits=bits, random=random, fresh=True, t=1, seed=8)
    for g in c.grads:
        g.zero_()
    old = [p.clone() for p in c.params]
    c.check()
    assert not c.m.float().any() and not c.v.float().any()
    for a, b in zip(c.params, old):
        assert ((a.double() - b.double() * (1 - 1e-3 * 0.05)).abs() <= 4 * U * b.abs()).all()


def test_small_roots_are_not_lost():
    """Elements far below their block's largest: the root stays above zero, so a step without a gradient is bounded."""
    for random in (False, True):
        c = Call([(256,)], bits=8, random=random, fresh=True, t=1, seed=9, factor=None, weight_decay=0.0)
        g = torch.full((256,), 1e-12, device=DEV)
        g[0] = 1.0
        c.grads = [g]
        c.check()
        assert (c.v.float() > 0).all()
        old = c.params[0].clone()
        c.grads = [torch.zeros(256, device=DEV)]
        c.step += 1
        c.check()
        # |m| / root is at most that of one gradient alone, sqrt of its corrections apart
        assert (c.params[0] - old).abs().max() <= 1e-3 * 1.5


def test_moments_too_small_for_their_units():
    c = Call([(512,)], bits=8, fresh=True, t=1, seed=10, factor=None)
    g = torch.full((512,), 1e-38, device=DEV)
    g[256:] = 1e-20
    c.grads = [g]
    c.run()
    torch.cuda.synchronize()
    assert not c.m[:256].float().any() and float(c.scales[0, 0]) == 0
    assert all(torch.isfinite(t.float()).all() for t in c.tensors())


def test_stochastic_rounding_has_the_right_mean():
    """One step from states of one value: of n elements a share of the root's fraction is rounded up, to the next value,
    within six standard deviations."""
    n = 1 << 16
    c = Call([(n,)], bits=8, random=True, fresh=True, t=5, seed=11, factor=None)
    c.m.zero_(), c.v.copy_(torch.full((n,), 16.0, device=DEV).to(torch.float8_e4m3fn))
    c.scales[:, 0], c.scales[:, 1] = 0, 1e-4
    g = torch.full((n,), 2e-3, device=DEV)
    g[::BLOCK] = 0.2   # the block's largest
    c.grads = [g]
    c.check()
    unit = float(c.scales[0, 1])
    q = math.sqrt(0.999 * 1.6e-3 ** 2 + 1e-3 * 2e-3 ** 2) / unit
    step = 2.0 ** (math.floor(math.log2(q)) - 3)
    up = q / step - math.floor(q / step)
    rest = torch.ones(n, dtype=torch.bool, device=DEV)
    rest[::BLOCK] = False
    held = c.v.float()[rest]
    assert set(held.unique().tolist()) == {math.floor(q / step) * step, (math.floor(q / step) + 1) * step}
    share = float((held > q).float().mean())
    assert abs(share - up) <= 6 * math.sqrt(up * (1 - up) / len(held))


def test_a_step_again_is_the_same_bits():
    for bits, random in STATES:
        a, b = (Call(bits=bits, random=random, seed=12) for _ in range(2))
        a.run(), b.run()
        assert all(torch.equal(x, y) for x, y in zip(a.bits(), b.bits()))


# ------------------------------------------------------------------- norm

def check_norm(grads, max_norm=1.0, **kw):
    want = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads if g is not None))
    out = ob.wtconv_grad_norm(grads, max_norm, **kw)
    factor = min(1.0, max_norm / (want + 1e-6))
    # sums in 64 bits, rounded once
    assert abs(float(out[0]) - want) <= 1.001 * U * want and abs(float(out[1]) - factor) <= 1.001 * U * factor
    return out


@pytest.mark.parametrize("shapes", [[(1,)], [(3,), (0,), (8,)], SHAPES, [((i * 91) % 3000,) for i in range(400)],
                                    [(20_000_003,)], [(17,)] * 161, [(8192,), (8193,), (2048 * 8192 + 5,)],
                                    [(2048,)] * 64, [(2047,), (131_072 - 2048,)], [(2049,)] * 32, [(2049,)] * 33, [(1,)] * 64,
                                    [(1,)] * 65, [(40_000,)] * 40, [(40_000,)] * 41])
def test_norm(shapes):
    g = torch.Generator(DEV).manual_seed(0)
    grads = [torch.randn(s, generator=g, device=DEV).to(F32 if i % 3 else BF16) for i, s in enumerate(shapes)]
    a = check_norm(grads)
    assert torch.equal(a, check_norm(grads))
    check_norm([x.bfloat16() for x in grads], 1e9)
    check_norm([None, *grads, None], math.inf)


def test_norm_of_far_values():
    for x in (1e-30, 1e-22, 1e18, 1e25):   # squares that 32 bits do not hold
        check_norm([torch.full((1000,), x, device=DEV), torch.full((9,), x, device=DEV).bfloat16()])
    assert ob.wtconv_grad_norm([torch.zeros(100, device=DEV)], 0.5).tolist() == [0.0, 1.0]
    assert ob.wtconv_grad_norm([torch.zeros(0, device=DEV)], 0.5).tolist() == [0.0, 1.0]


def test_norm_of_pointers_aligned_to_the_element_only():
    for t in (F32, BF16):
        check_norm([torch.randn(70_001, device=DEV).to(t)[1:], torch.randn(12, device=DEV).to(t)[3:]])


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_norm_that_is_not_finite_is_not_counted(bad):
    step = torch.full((1,), 4, dtype=torch.int64, device=DEV)
    grads = [torch.randn(5000, device=DEV), torch.randn(77, device=DEV).bfloat16()]
    check_norm(grads, step=step)
    assert int(step) == 5
    grads[1][50] = bad
    out = ob.wtconv_grad_norm(grads, 1.0, step=step)
    assert int(step) == 5 and not math.isfinite(float(out[0])) and math.isnan(float(out[1]))


def test_norm_into_given_tensors():
    out, ws = torch.empty(2, device=DEV), torch.full((1 << 16,), 255, dtype=torch.uint8, device=DEV)
    assert check_norm([torch.randn(999, device=DEV)], out=out, ws=ws) is out


# ------------------------------------------------------- streams and graphs

def test_on_another_stream():
    s = torch.cuda.Stream()
    c = Call(bits=8, seed=13)
    torch.cuda.synchronize()
    want = Step(*c.args(), **c.opts)
    norm = ob.wtconv_grad_norm(c.grads, 1.0, stream=s)
    c.run(stream=s)
    s.synchronize()
    want.check()
    assert torch.equal(norm, ob.wtconv_grad_norm(c.grads, 1.0))


def test_calls_at_once():
    """Steps and norms of other tensors on two streams at the same time."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [Call([(3_000_001,), (77,)], bits=8, random=True, seed=20 + i) for i in range(2)]
    alone = [Call([(3_000_001,), (77,)], bits=8, random=True, seed=20 + i) for i in range(2)]
    for _ in range(5):
        for c in alone:
            c.run()
    norms = [ob.wtconv_grad_norm(c.grads) for c in alone]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, s in zip(calls, streams):
            c.run(stream=s)
            got.append(ob.wtconv_grad_norm(c.grads, stream=s))
    torch.cuda.synchronize()
    for c, d in zip(calls, alone):
        assert all(torch.equal(x, y) for x, y in zip(c.bits(), d.bits()))
    assert all(torch.equal(g, norms[i % 2]) for i, g in enumerate(got))


@pytest.mark.parametrize("bits,random", STATES)
def test_captured_and_replayed(bits, random):
    """Norm and step in a graph: new gradients, counts, rates and random numbers are read at each replay."""
    shapes = [(300,), (40, 41), (9000,)] + [(50,)] * 100
    a, b = (Call(shapes, bits=bits, random=random, seed=14, t=0, lr_factor=1.0, factor=None) for _ in range(2))

    def step(c):
        norm = ob.wtconv_grad_norm(c.grads, 0.01, step=c.step)
        ob.wtconv_adamw_step(*c.args(), **{**c.opts, "factor": norm[1:]})
        return norm

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(a)
    torch.cuda.current_stream().wait_stream(s)
    step(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(a)
    for i in range(4):
        for x, y in zip(a.grads, b.grads):
            x.copy_(torch.randn(x.shape, device=DEV) * 1e-3)
            y.copy_(x)
        if i == 2:
            a.grads[1][3, 4] = b.grads[1][3, 4] = float("inf")   # skipped
        for c in (a, b):
            c.opts["lr_factor"].fill_(0.5 ** i)
            if random:
                c.opts["rng"][1] += 1
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(torch.nan_to_num(held, 7), torch.nan_to_num(step(b), 7))
        assert int(a.step) == int(b.step) == (2 + i if i < 2 else 1 + i)
        assert all(torch.equal(x, y) for x, y in zip(a.bits(), b.bits()))


# --------------------------------------------------------------- optimizer

def net(dtype=F32, seed=0):
    torch.manual_seed(seed)
    return torch.nn.Sequential(torch.nn.Linear(13, 37), torch.nn.GELU(), torch.nn.Linear(37, 5)).to(DEV, dtype)


def data(i, dtype=F32):
    g = torch.Generator(DEV).manual_seed(100 + i)
    return torch.randn(64, 13, generator=g, device=DEV).to(dtype), torch.randn(64, 5, generator=g, device=DEV).to(dtype)


def gradients(model, i):
    x, y = data(i, next(model.parameters()).dtype)
    model.zero_grad()
    ((model(x) - y) ** 2).mean().backward()


def test_optimizer_follows_torch():
    """The same updates as torch's own AdamW in 64 bits on the same gradients, two groups, clipped."""
    a = net()
    b = copy.deepcopy(a).double()
    groups = lambda m: [dict(params=[m[0].weight, m[2].weight], weight_decay=0.1),  # noqa: E731
                        dict(params=[m[0].bias, m[2].bias], weight_decay=0.0, lr=3e-3)]
    mine = AdamW(groups(a), lr=1e-2, eps=1e-6, betas=(0.8, 0.95), max_norm=0.05)
    other = torch.optim.AdamW(groups(b), lr=1e-2, eps=1e-6, betas=(0.8, 0.95))
    for i in range(20):
        gradients(a, i)
        for p, q in zip(a.parameters(), b.parameters()):
            q.grad = p.grad.double()
        torch.nn.utils.clip_grad_norm_(list(b.parameters()), 0.05)
        mine.step()
        other.step()
        for p, q in zip(a.parameters(), b.parameters()):
            # a step adds a few half steps of the parameter and 30 of the update (below 5 rates)
            assert (p.double() - q).abs().max() <= (i + 1) * U * (6 * q.abs().max() + 30 * 5e-2)
    assert int(mine._step) == 20


@pytest.mark.parametrize("dtype,master", [(F32, True), (BF16, True), (BF16, False)])
@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_state_round_trip(dtype, master, bits):
    """A run that is saved, loaded into a new optimizer and gone on with is the same run, bit for bit."""
    a = net(dtype)
    kw = dict(lr=1e-2, state_bits=bits, master=master, max_norm=1.0)
    mine = AdamW(a.parameters(), **kw)
    for i in range(3):
        gradients(a, i)
        mine.step()
    b = copy.deepcopy(a)
    saved = copy.deepcopy(mine.state_dict())
    theirs = AdamW(b.parameters(), **{**kw, "lr": 1.0})
    theirs.load_state_dict(saved)
    assert theirs.param_groups[0]["lr"] == 1e-2
    for i in range(3, 6):
        for m, o in ((a, mine), (b, theirs)):
            gradients(m, i)
            o.step()
        assert all(torch.equal(p, q) for p, q in zip(a.parameters(), b.parameters()))
    with pytest.raises(ValueError):
        AdamW(b.parameters(), **{**kw, "state_bits": 40 - bits}).load_state_dict(saved)
    with pytest.raises(ValueError):
        AdamW(list(b.parameters())[:2], **kw).load_state_dict(saved)


def test_optimizer_copies_and_files(tmp_path):
    """A copied optimizer goes on by itself; a state goes through a file that is read without executing anything."""
    a = net()
    o = AdamW(a.parameters(), state_bits=8, max_norm=1.0)
    gradients(a, 0)
    o.step()
    b, p = copy.deepcopy((a, o))
    assert p._buffers[0]["m"].data_ptr() != o._buffers[0]["m"].data_ptr() and p.max_norm == 1.0
    torch.save(o.state_dict(), tmp_path / "state.pt")
    c = copy.deepcopy(a)
    q = AdamW(c.parameters(), state_bits=8, max_norm=1.0)
    q.load_state_dict(torch.load(tmp_path / "state.pt", weights_only=True))
    for m, r in ((a, o), (b, p), (c, q)):
        gradients(m, 1)
        r.step()
    for x, y, z in zip(a.parameters(), b.parameters(), c.parameters()):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_master_copies_are_made_again():
    a = net(BF16)
    o = AdamW(a.parameters(), lr=1e-2)
    gradients(a, 0)
    o.step()
    other = net(BF16, seed=1)
    a.load_state_dict(other.state_dict())
    o.renew_master()
    for p, q in zip(a.parameters(), other.parameters()):
        p.grad = torch.zeros_like(p)
        q.grad = torch.zeros_like(q)
    o.param_groups[0]["lr"] = 0.0
    o.step()
    assert all(torch.equal(p, q) for p, q in zip(a.parameters(), other.parameters()))


def test_optimizer_groups_of_other_bits():
    """Large matrices in 8 bits, small vectors in 32: each group as an optimizer of its own."""
    a = net()
    b = copy.deepcopy(a)
    groups = lambda m: [dict(params=[m[0].weight, m[2].weight]), dict(params=[m[0].bias, m[2].bias], state_bits=32)]  # noqa: E731
    o = AdamW(groups(a), lr=1e-2, state_bits=8, rng=dropout_rng(4), site=9)
    p = [AdamW([groups(b)[0]], lr=1e-2, state_bits=8, rng=dropout_rng(4), site=9), AdamW([groups(b)[1]], lr=1e-2)]
    assert [x["state_bits"] for x in o.param_groups] == [8, 32]
    for i in range(3):
        for m, opts in ((a, [o]), (b, p)):
            gradients(m, i)
            for x in opts:
                x.step()
    assert [t.dtype for t in (o._buffers[0]["m"], o._buffers[1]["m"])] == [torch.float8_e4m3fn, F32]
    assert all(torch.equal(x, y) for x, y in zip(a.parameters(), b.parameters()))


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_groups_without_parameters(bits):
    """As when a list of parameters is split by a rule that holds for none or for all of them."""
    a, b = net(), net()
    mine = AdamW([dict(params=[]), dict(params=a.parameters()), dict(params=[], lr=0.5)], state_bits=bits, max_norm=1.0)
    plain = AdamW(b.parameters(), state_bits=bits, max_norm=1.0)
    for i in range(2):
        for m, o in ((a, mine), (b, plain)):
            gradients(m, i)
            o.step()
        mine.load_state_dict(copy.deepcopy(mine.state_dict()))
    assert all(torch.equal(p, q) for p, q in zip(a.parameters(), b.parameters()))


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_captured(bits):
    """A whole training step in a graph, against the same steps outside of one."""
    a, b = net(), net()
    rng = [dropout_rng(1) if bits == 8 else None for _ in range(2)]
    o, p = (AdamW(m.parameters(), lr=1e-2, state_bits=bits, max_norm=0.1, rng=r) for m, r in zip((a, b), rng))
    x, y = data(0)

    def step(m, opt):
        for w, g in zip(m.parameters(), torch.autograd.grad(((m(x) - y) ** 2).mean(), list(m.parameters()))):
            w.grad = g
        opt.step()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(a, o)
    torch.cuda.current_stream().wait_stream(s)
    step(b, p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, o)
    for i in range(1, 5):
        for t, n in zip((x, y), data(i)):
            t.copy_(n)
        for r in rng:
            if r is not None:
                r[1] += 1
        graph.replay()
        torch.cuda.synchronize()
        step(b, p)
        assert int(o._step) == int(p._step) == i + 1
        assert all(torch.equal(u, v) for u, v in zip(a.parameters(), b.parameters()))


@pytest.mark.parametrize("dtype,bits", [(F32, 32), (F32, 8), (BF16, 32)])
def test_a_captured_step_goes_on_from_a_loaded_state(dtype, bits):
    """The graph's buffers are those that the state is loaded into."""
    a = net(dtype)
    o = AdamW(a.parameters(), state_bits=bits, max_norm=0.1)
    for w in a.parameters():
        w.grad = torch.randn_like(w)
    o.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o.step()
    torch.cuda.synchronize()
    saved, weights = copy.deepcopy(o.state_dict()), copy.deepcopy(a.state_dict())
    results = []
    for _ in range(3):
        a.load_state_dict(weights)
        o.load_state_dict(saved)
        graph.replay()
        torch.cuda.synchronize()
        results.append(([w.detach().clone() for w in a.parameters()], copy.deepcopy(o.state_dict()["state"])))
        graph.replay()   # goes on, and is taken back
    assert int(results[0][1]["step"]) == 2
    first = results[0][1]["buffers"][0]
    for ws, st in results[1:]:
        assert all(torch.equal(p, q) for p, q in zip(ws, results[0][0]))
        assert int(st["step"]) == 2 and all(
            torch.equal(t.view(torch.uint8), first[k].view(torch.uint8)) for k, t in st["buffers"][0].items())
    assert not any(torch.equal(p, q) for p, q in zip(results[0][0], weights.values()))


def test_the_first_step_is_not_captured():
    """A graph would make the states again at every replay."""
    w = torch.nn.Parameter(torch.ones(300, device=DEV))
    w.grad = torch.ones_like(w)
    o = AdamW([w], max_norm=1.0)
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            o.step()
    assert torch.equal(w.detach(), torch.ones_like(w))
    o.step()
    assert int(o.state_dict()["state"]["step"]) == 1


def test_optimizer_skips_steps_that_are_not_finite():
    a = net()
    o = AdamW(a.parameters(), state_bits=8, max_norm=math.inf)
    gradients(a, 0)
    o.step()
    old = [p.clone() for p in a.parameters()]
    gradients(a, 1)
    a[0].bias.grad[2] = float("nan")
    o.step()
    assert all(torch.equal(p, q) for p, q in zip(a.parameters(), old)) and int(o._step) == 1
    assert math.isnan(float(o.last_norm[1]))
    gradients(a, 1)
    o.step()
    assert int(o._step) == 2 and not torch.equal(a[0].bias, old[1])


def test_optimizer_with_missing_and_strided_gradients():
    a = net()
    o = AdamW(a.parameters(), lr=0.1)
    gradients(a, 0)
    a[2].weight.grad = None
    a[0].weight.grad = a[0].weight.grad.t().contiguous().t()   # another memory order
    old = a[2].weight.clone()
    b = copy.deepcopy(a)
    b[0].weight.grad = a[0].weight.grad.contiguous()
    b[0].bias.grad, b[2].bias.grad = a[0].bias.grad, a[2].bias.grad
    o.step()
    AdamW(b.parameters(), lr=0.1).step()
    assert torch.equal(a[2].weight, old) and torch.equal(a[0].weight, b[0].weight)
    with pytest.raises(RuntimeError):
        o.add_param_group(dict(params=[torch.nn.Parameter(torch.zeros(3, device=DEV))]))


def test_a_change_in_place_is_seen_by_autograd():
    """A graph that needs the old parameter raises an error after the step."""
    a = net()
    o = AdamW(a.parameters())
    gradients(a, 0)
    x, _ = data(1)
    y = a(x.requires_grad_())
    o.step()
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


def test_refusals_on_the_gpu():
    c = Call([(40,), (5, 7)])
    p, g, m, v, t = c.args()
    kw = dict(c.opts)

    def call(p=p, g=g, m=m, v=v, t=t, **more):
        ob.wtconv_adamw_step(p, g, m, v, t, **{**kw, **more})

    big = torch.zeros(600, device=DEV)
    bad = [dict(p=[]), dict(g=g[:1]), dict(p=[p[0], p[1].bfloat16()]), dict(g=[g[0], g[1].bfloat16()]),
           dict(p=[p[0], p[1].double()], g=[g[0], g[1]]), dict(g=[g[0], g[1].t()]), dict(g=[g[0], g[1].reshape(7, 5)]),
           dict(p=[p[0], p[1].t()], g=[g[0], g[1].t().contiguous()]), dict(g=[g[0], g[1].cpu()]), dict(p=[p[0], p[1].cpu()]),
           dict(m=m[:256]), dict(m=m.double()), dict(v=big), dict(m=m.to(torch.float8_e4m3fn)), dict(t=None),
           dict(t=t.int()), dict(t=torch.ones(2, dtype=torch.int64, device=DEV)), dict(scales=torch.zeros(2, 2, device=DEV)),
           dict(master=m), dict(rng=torch.zeros(2, dtype=torch.int64, device=DEV)), dict(lr=[1e-3]), dict(lr=torch.ones(3)),
           dict(weight_decay=torch.ones(2, device=DEV)), dict(factor=torch.ones(2, device=DEV)), dict(site=-1),
           dict(factor=torch.ones(1, device=DEV).double()), dict(lr_factor=torch.ones(1)), dict(p=[p[0], "x"]), dict(site=1 << 31)]
    for i, kws in enumerate(bad):
        with pytest.raises(ValueError):
            call(**kws)
            pytest.fail(f"case {i}")
    for kws in (dict(p=[p[0], p[0]], g=[g[0], g[0]], m=m, v=v), dict(lr=float("nan")), dict(eps=0.0), dict(betas=(1.0, 0.9)),
                dict(v=m), dict(g=[p[0], g[1]])):
        with pytest.raises(RuntimeError):   # the library's own checks
            call(**kws)
    for i, args in enumerate(([], [torch.zeros(3)], [torch.zeros(3, device=DEV, dtype=torch.float16)],
                              [torch.zeros(4, 4, device=DEV).t()[:2]])):
        with pytest.raises(ValueError):
            ob.wtconv_grad_norm(args, 1.0)
    for kws in (dict(max_norm=0.0), dict(max_norm=float("nan")), dict(step=torch.zeros(1, device=DEV)),
                dict(out=torch.zeros(3, device=DEV))):
        with pytest.raises(ValueError):
            ob.wtconv_grad_norm(g, **kws)


# ------------------------------------------------------ as they are used together

@pytest.mark.parametrize("bits", [32, 8])
def test_a_block_with_experts_is_trained(bits):
    """Norm, experts, residual, backward pass, norm of the gradients and step: the gradients are those of the plain
    64-bit form, the step is the definition's."""
    B, H, W, C, E, K = 2, 5, 3, 24, 4, 2
    g = torch.Generator(DEV).manual_seed(0)
    p = {n: torch.nn.Parameter(0.3 * torch.randn(s, generator=g, device=DEV)) for n, s in
         dict(router=(E, C), up=(E, 2 * C, C), down=(E, C, 2 * C), gate=(C,), weight=(C,), bias=(C,)).items()}
    x = torch.randn(B, C, H, W, generator=g, device=DEV)
    dy = torch.randn(B, C, H, W, generator=g, device=DEV)

    def block(p, x, plain, expert=None):
        if plain:
            z = (x - x.mean(1, keepdim=True)) / (x.var(1, correction=0, keepdim=True) + 1e-6).sqrt()
            u = (z * p["weight"].view(-1, 1, 1) + p["bias"].view(-1, 1, 1)).permute(0, 2, 3, 1)
        else:
            u = channel_norm(x, p["weight"], p["bias"], channels_last=True).permute(0, 2, 3, 1)
        logits = u @ p["router"].t()
        if expert is None:
            expert = logits.topk(K, -1)[1]
        w = torch.softmax(logits.gather(-1, expert), -1)
        if plain:
            # every expert on every row, and the chosen ones of them
            each = torch.stack([torch.tanh(u @ p["up"][e].t()) @ p["down"][e].t() for e in range(E)], -2)
            h = (each.gather(-2, expert.unsqueeze(-1).expand(*expert.shape, C)) * w.unsqueeze(-1)).sum(-2)
            return x + p["gate"].view(-1, 1, 1) * h.permute(0, 3, 1, 2), expert
        route = expert_sort(expert, E)
        rows = expert_rows(u, route)
        ends = route.offsets.tolist()
        ys = torch.cat([torch.tanh(rows[a:b] @ p["up"][e].t()) @ p["down"][e].t()
                        for e, (a, b) in enumerate(zip(ends, ends[1:]))])
        h = expert_sum(ys, w, route).permute(0, 3, 1, 2)
        return block_residual(x, h, gate=p["gate"]), expert

    o = AdamW(p.values(), lr=1e-2, state_bits=bits, max_norm=1.0, rng=dropout_rng(3) if bits == 8 else None, site=50)
    for i in range(4):
        o.zero_grad()
        y, expert = block(p, x, False)
        y.backward(dy)
        q = {n: t.detach().double().requires_grad_() for n, t in p.items()}
        z, _ = block(q, x.double(), True, expert)
        z.backward(dy.double())
        assert (y.double() - z).abs().max() <= 1e-5 * z.abs().max()
        for n in p:   # sums of hundreds of fp32 terms
            assert (p[n].grad.double() - q[n].grad).abs().max() <= 2e-5 * q[n].grad.abs().max(), n
        if i:
            b = o._buffers[0]
            factor = ob.wtconv_grad_norm([t.grad for t in p.values()], 1.0)[1:]
            want = Step(list(p.values()), [t.grad for t in p.values()], b["m"], b["v"], int(o._step) + 1, lr=1e-2,
                        weight_decay=1e-2, scales=b.get("scales"), factor=factor, rng=o.rng, site=50)
            o.step()
            want.check()
        else:
            o.step()
        if o.rng is not None:
            o.rng[1] += 1


# ------------------------------------------------------------ refused steps

def _state(model, o):
    return ([p.detach().clone() for p in model.parameters()], None if o._step is None else int(o._step),
            [None if b is None else {k: t.clone() for k, t in b.items()} for b in o._buffers])


def _same_state(a, b):
    return (all(torch.equal(x, y) for x, y in zip(a[0], b[0])) and a[1] == b[1]
            and all(x is y or all(torch.equal(x[k].view(torch.uint8), y[k].view(torch.uint8)) for k in x)
                    for x, y in zip(a[2], b[2])))


# what is wrong in the second group, or for all: how it comes, and how it goes
REFUSED = {
    "rate": (lambda o, q: o.param_groups[1].update(lr=float("nan")), lambda o, q: o.param_groups[1].update(lr=1e-2)),
    "decay": (lambda o, q: o.param_groups[1].update(weight_decay=math.inf),
              lambda o, q: o.param_groups[1].update(weight_decay=1e-2)),
    "eps": (lambda o, q: o.param_groups[1].update(eps=1e-40), lambda o, q: o.param_groups[1].update(eps=1e-8)),
    "betas": (lambda o, q: o.param_groups[1].update(betas=(0.9, 1.0)),
              lambda o, q: o.param_groups[1].update(betas=(0.9, 0.999))),
    "rng": (lambda o, q: setattr(o, "rng", o.rng.repeat(2)), lambda o, q: setattr(o, "rng", o.rng[:2].clone())),
    "lr_factor": (lambda o, q: setattr(o, "lr_factor", torch.ones(2, device=DEV)), lambda o, q: setattr(o, "lr_factor", None)),
    "site": (lambda o, q: setattr(o, "site", 2 ** 31 - 1), lambda o, q: setattr(o, "site", 40)),
    "norm": (lambda o, q: setattr(o, "max_norm", -1.0), lambda o, q: setattr(o, "max_norm", 1.0)),
    "its own gradient": (lambda o, q: setattr(q, "grad", q.data), lambda o, q: setattr(q, "grad", torch.full_like(q, 0.1))),
}


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("what", REFUSED)
def test_a_refused_step_leaves_everything_as_it_was(what, first):
    """The count, the states and the groups before the one that is wrong; once it is right the step is the one that
    an optimizer takes to which that did not happen."""
    wrong, right = REFUSED[what]
    models = net(), net()
    opts = [AdamW([dict(params=[m[0].weight, m[0].bias]), dict(params=[m[2].weight, m[2].bias])], lr=1e-2, state_bits=8,
                  max_norm=1.0, rng=dropout_rng(5), site=40) for m in models]
    if not first:
        for m, o in zip(models, opts):
            gradients(m, 0)
            o.step()
    for m in models:
        gradients(m, 1)
        m[2].bias.grad = torch.full_like(m[2].bias, 0.1)
    (a, b), (o, p) = models, opts
    before = _state(a, o)
    wrong(o, a[2].bias)
    for _ in range(2):
        with pytest.raises((ValueError, RuntimeError)):
            o.step()
        torch.cuda.synchronize()
        assert _same_state(before, _state(a, o))
    right(o, a[2].bias)
    for x in opts:
        x.step()
    assert _same_state(_state(a, o), _state(b, p)) and int(o._step) == (1 if first else 2)


def test_a_refused_first_step_makes_no_master_copies():
    """They are made from the parameters as they are at the first step that is taken."""
    a = net(BF16)
    o = AdamW(a.parameters(), lr=1e-2)
    o.param_groups[0]["lr"] = float("inf")
    gradients(a, 0)
    with pytest.raises(RuntimeError):
        o.step()
    assert o._step is None and o._buffers == [None]
    b = net(BF16, seed=1)
    a.load_state_dict(b.state_dict())
    o.param_groups[0]["lr"] = 1e-2
    p = AdamW(b.parameters(), lr=1e-2)
    for m, x in ((a, o), (b, p)):
        gradients(m, 2)
        x.step()
    assert all(torch.equal(u, v) for u, v in zip(a.parameters(), b.parameters()))


@pytest.mark.parametrize("kind", ["tensor", "tensor of 64 bits", "numpy"])
def test_rates_that_are_not_python_s_numbers(kind):
    """A rate or decay that a scheduler holds as a tensor on the host, or as numpy's number."""
    import numpy as np

    make = {"tensor": torch.tensor, "tensor of 64 bits": lambda x: torch.tensor([x], dtype=torch.float64),
            "numpy": np.float32}[kind]
    models = net(), net()
    opts = [AdamW(m.parameters(), lr=f(1e-2), weight_decay=f(0.25)) for m, f in zip(models, (make, float))]
    for i, rate in enumerate((1e-2, 0.5, 0.0)):
        for m, o, f in zip(models, opts, (make, float)):
            o.param_groups[0]["lr"] = f(rate)
            gradients(m, i)
            o.step()
        assert all(torch.equal(torch.tensor(float(x.param_groups[0]["lr"])), torch.tensor(rate)) for x in opts)
        assert all(torch.equal(p, q) for p, q in zip(*(m.parameters() for m in models)))
    before = _state(models[0], opts[0])
    opts[0].param_groups[0]["lr"] = torch.ones((), device=DEV)
    gradients(models[0], 3)
    with pytest.raises(ValueError, match="lr_factor"):
        opts[0].step()
    assert _same_state(before, _state(models[0], opts[0]))


def test_rounding_is_not_the_dropouts_bits():
    """With the rng that the model's dropouts take, at the offset of this step, and no site given."""
    rng = dropout_rng(3)
    params = [torch.nn.Parameter(torch.randn(700, device=DEV)) for _ in range(3)]
    o = AdamW(params, lr=1e-3, state_bits=8, rng=rng)
    for i in range(2):
        for q in params:
            q.grad = torch.randn(700, device=DEV) * 1e-2
        if i:
            b, copies = o._buffers[0], [q.detach().clone() for q in params]
            args = [copies, [q.grad for q in params], b["m"], b["v"], int(o._step) + 1]
            kw = dict(lr=1e-3, weight_decay=1e-2, scales=b["scales"], rng=rng)
            want, other = Step(*args, **kw, site=1 << 30), Step(*args, **kw, site=0)
        o.step()
        rng[1] += 1
    rng[1] -= 1
    for q, c in zip(params, copies):
        c.copy_(q.detach())
    want.check()
    with pytest.raises(AssertionError):
        other.check()


def test_refusals_on_another_stream():
    """They are the same as on the current one."""
    c, s = Call([(40,), (5, 7)], bits=8), torch.cuda.Stream()
    p, g, m, v, t = c.args()
    for stream in (None, s):
        for args, kw in (((p, [g[0], g[1].cpu()], m, v, t), {}), ((p, g, m.cpu(), v, t), {}), ((p, g, m, v, t.cpu()), {}),
                         ((p, g, m, v, t), dict(factor=torch.ones(1))), ((p, g, m, v, t), dict(rng=torch.zeros(2, dtype=torch.int64))),
                         (([p[0].cpu(), p[1]], g, m, v, t), {}), ((["x", p[1]], g, m, v, t), {}), ((p, ["x", None], m, v, t), {}),
                         ((p, g, m, v, 3), {}), (([], [], m, v, t), {})):
            with pytest.raises(ValueError):
                ob.wtconv_adamw_step(*args, **{**c.opts, **kw}, stream=stream)
        for args, kw in (([g[0].cpu()], {}), ([g[0], g[1].cpu()], {}), (["x"], {}), ([None], {}), ([g[0]], dict(out=torch.zeros(2))),
                         ([g[0]], dict(step=torch.zeros(1, dtype=torch.int64))), ([g[0]], dict(ws=5))):
            with pytest.raises(ValueError):
                ob.wtconv_grad_norm(args, 1.0, **kw, stream=stream)


def test_states_and_outputs_are_seen_by_autograd():
    """What a step and a norm write counts as changed in place; what they do not, not."""
    c = Call([(40,), (300,)], p=BF16, master=True, bits=8, missing=(1,))
    out = torch.empty(2, device=DEV)
    written = [c.params[0], c.m, c.v, c.scales, c.master]
    others = [c.params[1], c.grads[0], c.step]
    before = [t._version for t in written + others]
    c.run()
    assert [t._version for t in written + others] == [n + (i < len(written)) for i, n in enumerate(before)]
    before = c.step._version, c.grads[0]._version, out._version
    ob.wtconv_grad_norm(c.grads, 1.0, step=c.step, out=out)
    assert (c.step._version, c.grads[0]._version, out._version) == (before[0] + 1, before[1], before[2] + 1)


# around a wavefront's blocks and a workgroup's piece, of 1,024 or 2,048 elements by types and states
PIECES = [(1023,), (1024,), (1025,), (2047,), (2048,), (2049,), (4095,), (4096,), (1,), (3 * 2048 + 5,)]


@pytest.mark.parametrize("bits,random", STATES)
@pytest.mark.parametrize("p,g,master", KINDS)
def test_sizes_around_a_workgroup_s_piece(p, g, master, bits, random):
    Call(PIECES, p=p, g=g, master=master, bits=bits, random=random, seed=21).check()


# the largest tensor of a call, and one beyond 2^32 elements whose states are in 32 bits: grids of more than one row
@pytest.mark.parametrize("p,bits,n,gib", [(BF16, 8, 2 ** 34, 150), (F32, 32, 2 ** 32 + 5001, 110)])
def test_the_largest_tensor(p, bits, n, gib, monkeypatch):
    """All of it holds the same numbers, but for windows, which hold others: the windows are those of the 64-bit form,
    and everything else is alike afterwards. A small tensor stands behind it."""
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB")
    import numpy as np

    import tests._step_ref as ref
    from tests._block_ref import philox

    gen = torch.Generator(DEV).manual_seed(n % 1009)
    kind = torch.float8_e4m3fn if bits == 8 else F32
    whole = -(-n // BLOCK) * BLOCK
    P, G = torch.full((n,), 0.5, dtype=p, device=DEV), torch.full((n,), 2.0 ** -16, dtype=p, device=DEV)
    P2, G2 = torch.randn(300, generator=gen, device=DEV).to(p), torch.randn(300, generator=gen, device=DEV).to(p)
    m, v = (torch.zeros(whole + 512, dtype=kind, device=DEV) for _ in range(2))
    scales = torch.zeros((whole + 512) // BLOCK, 2, device=DEV) if bits == 8 else None
    rng = dropout_rng(5) if bits == 8 else None
    step = torch.ones(1, dtype=torch.int64, device=DEV)
    kw = dict(lr=1e-2, weight_decay=0.1)
    windows = [slice(a, min(n, a + 1024)) for a in (1024, 2 ** 30 - 512, 2 ** 31 - 512, 2 ** 32 - 512,
                                                    n // BLOCK * BLOCK - 1024, n // BLOCK * BLOCK - 256)]
    windows[-2] = slice(windows[-2].start, windows[-1].start)
    real = ref.random_bits

    def bits_from(first):
        def window(count, tensor, site, rng):
            seed, offset = (int(x) & (2 ** 64 - 1) for x in rng.tolist())
            groups = np.arange(first // 4, first // 4 - (-count // 4))
            words = philox(groups, site + tensor, offset, seed).reshape(-1)[:count].astype(np.int64)
            return torch.from_numpy(np.stack([words & 0xFFFF, words >> 16], -1)).double()
        return window

    wants = []
    for w in windows:
        k = w.stop - w.start
        P[w], G[w] = torch.randn(k, generator=gen, device=DEV).to(p), (1e-3 * torch.randn(k, generator=gen, device=DEV)).to(p)
        states = slice(w.start, w.start + -(-k // BLOCK) * BLOCK)
        wants.append(Step([P[w]], [G[w]], m[states], v[states], 1, **kw, rng=rng, site=9,
                          scales=None if scales is None else scales[states.start // BLOCK:states.stop // BLOCK]))
    wants.append(Step([P2], [G2], m[whole:], v[whole:], 1, **kw, rng=rng, site=10,
                      scales=None if scales is None else scales[whole // BLOCK:]))
    rest = n - sum(w.stop - w.start for w in windows)
    squares = rest * 2.0 ** -32 + sum(float((G[w].double() ** 2).sum()) for w in windows) + float((G2.double() ** 2).sum())
    norm = ob.wtconv_grad_norm([G, G2], math.inf)
    ob.wtconv_adamw_step([P, P2], [G, G2], m, v, step, **kw, scales=scales, rng=rng, site=9)
    torch.cuda.synchronize()
    assert abs(float(norm[0]) - math.sqrt(squares)) <= 1.001 * U * math.sqrt(squares)
    for w, want in zip(windows, wants):
        monkeypatch.setattr(ref, "random_bits", bits_from(w.start))
        want.check()
    monkeypatch.setattr(ref, "random_bits", real)
    wants[-1].check()
    # everything else: the element before the first window's
    alike = [P[0].clone(), m[0].clone().view(torch.uint8 if bits == 8 else F32), v[0].clone().view(torch.uint8 if bits == 8 else F32)]
    assert float(P[0]) < 0.5 and float(m[0].float()) > 0 and float(v[0].float()) > 0
    for at in range(0, n, 2 ** 30):
        end = min(n, at + 2 ** 30)
        other = torch.zeros(end - at, dtype=torch.bool, device=DEV)
        for t, one in zip((P, m.view(alike[1].dtype), v.view(alike[2].dtype)), alike):
            other |= t[at:end] != one
        for w in windows:
            a, b = max(w.start, at), min(w.stop, end)
            if a < b:
                other[a - at:b - at] = False
        assert not other.any(), (at, other.nonzero()[:4])
    if scales is not None:
        blocks = torch.ones(n // BLOCK, dtype=torch.bool, device=DEV)
        for w in windows:
            blocks[w.start // BLOCK:-(-w.stop // BLOCK)] = False
        assert (scales[:n // BLOCK][blocks] == scales[0]).all()
    del P, G, m, v, scales, other, wants
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", [list, tuple, torch.tensor])
def test_a_rate_for_each_parameter_of_a_group(kind):
    """Rates and decays set as a sequence, or a tensor on the host, are those of groups of one parameter each."""
    a, b = net(), net()
    rates, decays = [1e-2, 3e-3, 5e-2, 0.0], [0.0, 0.1, 0.2, 0.3]
    o = AdamW(a.parameters(), max_norm=1.0)
    o.param_groups[0].update(lr=kind(rates), weight_decay=kind(decays))
    p = AdamW([dict(params=[q], lr=r, weight_decay=d) for q, r, d in zip(b.parameters(), rates, decays)], max_norm=1.0)
    for i in range(3):
        for m, x in ((a, o), (b, p)):
            gradients(m, i)
            x.step()
    assert all(torch.equal(x, y) for x, y in zip(a.parameters(), b.parameters()))
    before = _state(a, o)
    o.param_groups[0]["lr"] = kind(rates[:3])
    with pytest.raises(ValueError):
        o.step()
    assert _same_state(before, _state(a, o))
