"""The 64-bit forms that the expert rows and the optimizer's step are held to, against other ways to the same (CPU)."""
import math

import pytest
import torch

from tests._step_ref import BLOCK, Step, check_codes, e4m3_steps, random_bits, rows_ref, sort_ref, sum_bwd_ref, sum_ref


def test_nearest_numbers_are_those_of_the_type():
    q = torch.cat([torch.randn(4000, dtype=torch.float64) * s for s in (1e-3, 0.02, 1.0, 100.0)]).clamp(-448, 448)
    got = q.float().to(torch.float8_e4m3fn).double()
    check_codes("torch", got, q, torch.full_like(q, 1e-7) * q.abs(), torch.ones_like(q), None)
    with pytest.raises(AssertionError):   # a number of the type that is not the nearest
        check_codes("off", got + e4m3_steps(q), q, 1e-7 * q.abs(), torch.ones_like(q), None)


def test_random_bits_choose_the_neighbours_in_the_right_shares():
    q = torch.full((60_000,), 1.30, dtype=torch.float64)   # between 1.25 and 1.375
    u = random_bits(60_000, 3, 7, torch.tensor([11, 12]))[:, 0]
    held = torch.floor(q / 0.125 + (u + 0.5) / 65536) * 0.125
    check_codes("random", held, q, 0 * q, torch.ones_like(q), u)
    assert set(held.unique().tolist()) == {1.25, 1.375}
    share = float((held > 1.3).double().mean())
    assert abs(share - 0.4) <= 6 * math.sqrt(0.4 * 0.6 / 60_000)
    with pytest.raises(AssertionError):
        check_codes("other bits", held, q, 0 * q, torch.ones_like(q), u.flip(0))


def test_routing_forms():
    e = torch.tensor([[2, 0], [-1, 2], [0, 5], [2, 2]])
    order, place, offsets = sort_ref(e, 3)
    assert order.tolist() == [1, 4, 0, 3, 6, 7, 2, 5] and offsets.tolist() == [0, 2, 2, 6]
    assert place.tolist() == [[2, 0], [6, 3], [1, 7], [4, 5]]
    place, offsets = torch.tensor(place), torch.tensor(offsets)
    x = torch.randn(4, 3)
    xs, written = rows_ref(x, place, offsets)
    assert torch.equal(xs[:6], x[[0, 2, 0, 1, 3, 3]]) and not xs[6:].any() and written.all()
    w = torch.rand(4, 2)
    ys = torch.randn(8, 3, dtype=torch.float64, requires_grad=True)
    wd = w.double().requires_grad_()
    live = torch.tensor([[1, 1], [0, 1], [1, 0], [1, 1]])
    y = torch.stack([sum(live[n, k] * wd[n, k] * ys[place[n, k]] for k in range(2)) for n in range(4)])
    assert (sum_ref(ys.detach().float(), w, place, offsets)[0] - y).abs().max() <= 1e-6
    dy = torch.randn(4, 3)
    dys, dw = torch.autograd.grad(y, (ys, wd), dy.double())
    want = sum_bwd_ref(dy, ys.detach().float(), w, place, offsets)
    assert (want[0][0] - dys).abs().max() <= 1e-6 and (want[1][0] - dw).abs().max() <= 1e-6


def test_step_form_is_torch_s_adamw():
    """torch's own AdamW in 32 bits passes the check of a step; a step with another rate, a forgotten correction or a
    changed gap between tensors does not."""
    torch.manual_seed(0)
    params = [torch.randn(s) for s in ((7, 5), (300,))]
    n = 256 + 512

    def call(lr=1e-2, t=3, gap=False):
        ps = [p.clone() for p in params]
        grads = [torch.randn(p.shape) for p in ps]
        m, v = torch.zeros(n), torch.zeros(n)
        at = [slice(0, 35), slice(256, 556)]
        q = [torch.nn.Parameter(p.clone()) for p in ps]
        o = torch.optim.AdamW(q, lr=lr, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
        for x, s in zip(q, at):
            m[s], v[s] = 0.1 * torch.randn(x.numel()), torch.rand(x.numel())
            o.state[x] = {"step": torch.tensor(float(t - 1)), "exp_avg": m[s].view(x.shape).clone(),
                          "exp_avg_sq": v[s].view(x.shape).clone()}
        want = Step(ps, grads, m, v, 3, lr=1e-2, weight_decay=0.1, betas=(0.9, 0.99), eps=1e-6)
        for x, g in zip(q, grads):
            x.grad = g
        o.step()
        for x, p, s in zip(q, ps, at):
            p.copy_(x.detach())
            m[s], v[s] = o.state[x]["exp_avg"].view(-1), o.state[x]["exp_avg_sq"].view(-1)
        if gap:
            m[100] = 1
        want.check()

    call()
    for kw in (dict(lr=1.001e-2), dict(t=4), dict(gap=True)):
        with pytest.raises(AssertionError):
            call(**kw)
    assert BLOCK == 256
