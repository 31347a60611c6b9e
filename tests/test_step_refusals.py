"""What the expert rows and the optimizer's step refuse before anything is launched (CPU)."""
import ctypes
import os

import pytest
import torch

from wavelet_convolution_amd import binding as wt
from wavelet_convolution_amd import expert_binding as eb
from wavelet_convolution_amd import experts as ex
from wavelet_convolution_amd import optim as op
from wavelet_convolution_amd import optim_binding as ob

P = [ctypes.c_void_p((i + 1) << 40) for i in range(10)]   # never dereferenced: validation fails first
NONE = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(wt._LIB_PATH):
        pytest.skip("libwtconv.so not built")
    return wt.load_library()


def _d(**kw):
    d = dict(n=100, k=2, experts=8, c=16, dtype=0)
    d.update(kw)
    return ctypes.byref(wt.WTConvExpertDesc(**d))


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(k=0), 1), (dict(k=-2), 1), (dict(experts=0), 1), (dict(k=1025), 2), (dict(experts=1025), 2),
    (dict(n=1 << 31, k=1), 2), (dict(n=1 << 30, k=2), 2), (dict(n=1 << 62, k=1024), 2)])
def test_bad_routings(lib, kw, status):
    assert lib.wtconv_expert_workspace_size(_d(**kw)) == NONE
    assert lib.wtconv_expert_sort(_d(**kw), P[0], 0, P[1], P[2], P[3], P[4], 1 << 30, None) == status
    for fn in (lib.wtconv_expert_rows_fwd, lib.wtconv_expert_rows_bwd):
        assert fn(_d(**kw), P[0], P[1], P[2], P[3], None) == status
    assert lib.wtconv_expert_sum_fwd(_d(**kw), *P[:5], None) == status
    assert lib.wtconv_expert_sum_bwd(_d(**kw), *P[:7], None) == status


@pytest.mark.parametrize("kw,status", [(dict(c=0), 1), (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(c=(1 << 30) + 1), 2),
                                       (dict(n=1 << 20, k=1, c=1 << 30), 2)])
def test_bad_rows(lib, kw, status):
    for fn in (lib.wtconv_expert_rows_fwd, lib.wtconv_expert_rows_bwd):
        assert fn(_d(**kw), P[0], P[1], P[2], P[3], None) == status
    assert lib.wtconv_expert_sum_fwd(_d(**kw), *P[:5], None) == status
    assert lib.wtconv_expert_sum_bwd(_d(**kw), *P[:7], None) == status


def test_bad_pointers_of_a_sort(lib):
    def sort(d=_d(), expert=P[0], ids=1, order=P[1], place=P[2], offsets=P[3], ws=None, n=0):
        return lib.wtconv_expert_sort(d, expert, ids, order, place, offsets, ws, n, None)

    assert lib.wtconv_expert_sort(None, P[0], 0, *P[1:4], None, 0, None) == 1
    at = ctypes.c_void_p
    for kw in (dict(expert=None), dict(order=None), dict(place=None), dict(offsets=None), dict(ids=2), dict(ids=-1),
               dict(expert=at((1 << 40) + 4)), dict(order=at((1 << 41) + 2)), dict(order=P[0]), dict(place=P[1]),
               dict(offsets=at((1 << 40) + 796)), dict(place=at((2 << 40) + 796)), dict(ws=P[1], n=4096)):
        assert sort(**kw) == 1, kw
    assert lib.wtconv_expert_workspace_size(_d()) == 0
    big = _d(n=100_000)
    need = lib.wtconv_expert_workspace_size(big)
    assert 0 < need < 1 << 20
    assert sort(big) == 3 and sort(big, ws=P[4], n=need - 1) == 3 and sort(big, ws=at((5 << 40) + 64), n=1 << 20) == 3


def test_bad_pointers_of_rows(lib):
    at = ctypes.c_void_p
    for fn in (lib.wtconv_expert_rows_fwd, lib.wtconv_expert_rows_bwd):
        ok = [_d(), *P[:4], None]
        for i in range(1, 5):
            assert fn(*[None if j == i else a for j, a in enumerate(ok)]) == 1
        assert fn(_d(), at((1 << 40) + 2), *P[1:4], None) == 1 and fn(_d(), P[0], P[1], P[2], P[0], None) == 1
        assert fn(_d(), P[0], P[1], P[2], at((2 << 40) + 8), None) == 1
        assert fn(_d(dtype=1), at((1 << 40) + 1), *P[1:4], None) == 1
        assert fn(_d(n=0), *[None] * 4, None) == 0
    for i in range(5):
        assert lib.wtconv_expert_sum_fwd(_d(), *[None if j == i else p for j, p in enumerate(P[:5])], None) == 1
    assert lib.wtconv_expert_sum_fwd(_d(), *P[:4], P[1], None) == 1
    call = lambda *a: lib.wtconv_expert_sum_bwd(_d(), *a, None)  # noqa: E731
    dy, ys, w, place, offsets, dys, dw = P[:7]
    assert call(dy, ys, w, place, offsets, None, None) == 0   # nothing is wanted
    for bad in ((None, ys, w, place, offsets, dys, dw), (dy, None, w, place, offsets, dys, dw),
                (dy, ys, None, place, offsets, dys, dw), (dy, ys, w, None, offsets, dys, dw),
                (dy, ys, w, place, None, dys, dw), (dy, ys, w, place, offsets, dy, dw),
                (dy, ys, w, place, offsets, ys, dw), (dy, ys, w, place, offsets, dys, dys),
                (dy, ys, w, place, offsets, dys, w)):
        assert call(*bad) == 1


def test_host_tensors_are_refused():
    x, place, offsets = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    ys, w = torch.zeros(8, 8), torch.zeros(4, 2)
    route = ex.ExpertRoute(place.view(-1), place, offsets)
    for call in (lambda: eb.wtconv_expert_sort(place, 2), lambda: eb.wtconv_expert_rows_fwd(x, place, offsets),
                 lambda: eb.wtconv_expert_rows_bwd(ys, place, offsets),
                 lambda: eb.wtconv_expert_sum_fwd(ys, w, place, offsets),
                 lambda: eb.wtconv_expert_sum_bwd(x, ys, w, place, offsets), lambda: ob.wtconv_grad_norm([x]),
                 lambda: ob.wtconv_adamw_step([x], [x.clone()], torch.zeros(256), torch.zeros(256),
                                              torch.ones(1, dtype=torch.int64), lr=1e-3, weight_decay=0.0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ex.expert_sort(place, 2), lambda: ex.expert_rows(x, route),
                 lambda: ex.expert_sum(ys, w, route)):
        with pytest.raises(RuntimeError, match="GPU only"):
            call()


# ---------------------------------------------------------------- AdamW

def _arrays(counts, params, grads, lr=1e-3, wd=0.0):
    n = len(counts)
    return ((ctypes.c_void_p * n)(*params), (ctypes.c_void_p * n)(*grads), (ctypes.c_int64 * n)(*counts),
            (ctypes.c_float * n)(*[lr] * n), (ctypes.c_float * n)(*[wd] * n))


def _adamw(lib, counts=(1000, 300), params=(1 << 40, 2 << 40), grads=(3 << 40, 4 << 40), lr=1e-3, wd=0.0, m=5 << 40,
           v=6 << 40, scales=None, master=None, step=7 << 40, factor=None, lr_factor=None, rng=None, n=None, **kw):
    d = dict(p_dtype=0, g_dtype=0, state_bits=32, site=0, beta1=0.9, beta2=0.999, eps=1e-8)
    d.update(kw)
    a = _arrays(counts, params, grads, lr, wd)
    return lib.wtconv_adamw_step(ctypes.byref(wt.WTConvAdamWDesc(**d)), len(counts) if n is None else n, *a, m, v,
                                 scales, master, step, factor, lr_factor, rng, None)


@pytest.mark.parametrize("kw,status", [
    (dict(p_dtype=2), 1), (dict(g_dtype=-1), 1), (dict(state_bits=16), 1), (dict(beta1=1.0), 1), (dict(beta2=-0.1), 1),
    (dict(beta1=float("nan")), 1), (dict(eps=0.0), 1), (dict(eps=1e-40), 1), (dict(eps=float("inf")), 1), (dict(n=-1), 1),
    (dict(m=None), 1), (dict(v=None), 1), (dict(step=None), 1), (dict(lr=float("nan")), 1), (dict(wd=float("inf")), 1),
    (dict(scales=8 << 40), 1), (dict(state_bits=8), 1), (dict(master=8 << 40), 1), (dict(rng=8 << 40), 1),
    (dict(state_bits=8, scales=8 << 40, rng=9 << 40, site=-1), 1),
    (dict(state_bits=8, scales=8 << 40, rng=9 << 40, site=(1 << 31) - 1), 1),
    (dict(counts=(1000, -1)), 2), (dict(counts=(1000, (1 << 34) + 1)), 2), (dict(counts=(1 << 34,) * 33, params=[1] * 33, grads=[1] * 33), 2),
    (dict(params=(None, 2 << 40)), 1), (dict(params=((1 << 40) + 2, 2 << 40)), 1), (dict(grads=((3 << 40) + 2, 4 << 40)), 1),
    (dict(m=(5 << 40) + 8), 1), (dict(v=(6 << 40) + 4), 1), (dict(step=(7 << 40) + 4), 1), (dict(factor=(8 << 40) + 2), 1),
    (dict(lr_factor=(8 << 40) + 1), 1),
    # the same tensor twice, and overlaps of outputs with each other and with inputs
    (dict(params=(1 << 40, 1 << 40)), 1), (dict(params=(1 << 40, (1 << 40) + 3996)), 1), (dict(grads=(1 << 40, 4 << 40)), 1),
    (dict(grads=(3 << 40, (1 << 40) + 2000)), 1), (dict(v=5 << 40), 1), (dict(v=(5 << 40) + 1296 * 4), 1), (dict(m=2 << 40), 1),
    (dict(step=(5 << 40) + 8), 1), (dict(factor=2 << 40), 1),
])
def test_bad_steps(lib, kw, status):
    assert _adamw(lib, **kw) == status


def test_steps_of_nothing(lib):
    assert _adamw(lib, counts=(), params=(), grads=()) == 0
    assert _adamw(lib, counts=(0, 5), grads=(3 << 40, None)) == 0          # nothing to do: nothing is launched
    assert lib.wtconv_adamw_step(None, 0, *[None] * 14) == 1


def test_state_count(lib):
    def count(*c):
        return lib.wtconv_adamw_state_count((ctypes.c_int64 * len(c))(*c), len(c))

    assert count() == 0 and count(0) == 0 and count(1) == 256 and count(256) == 256 and count(257, 1, 0, 512) == 1280
    assert count(1 << 34) == 1 << 34 and count((1 << 34) + 1) == -1 and count(-1) == -1
    assert count(*[1 << 34] * 32) == 1 << 39 and count(*[1 << 34] * 32, 1) == -1
    assert lib.wtconv_adamw_state_count(None, 1) == -1 and lib.wtconv_adamw_state_count(None, -1) == -1


def test_bad_norms(lib):
    def size(*counts):
        return lib.wtconv_grad_norm_workspace_size((ctypes.c_int64 * len(counts))(*counts), len(counts))

    need = size(200_000, 50)
    assert 0 < need < 1 << 16 and lib.wtconv_grad_norm_workspace_size(None, -1) == NONE
    assert size() == size(100, 0, 2048) == size(*[1] * 64) == 0 < size(*[1] * 65)
    assert size(-1) == size((1 << 34) + 1) == lib.wtconv_grad_norm_workspace_size(None, 2) == NONE
    assert size(*[10_000] * 1000) >= 8 * 1000

    def norm(counts=(200_000, 50), grads=(1 << 40, 2 << 40), dtypes=(0, 1), max_norm=1.0, step=None, out=3 << 40, ws=4 << 40,
             bytes_=need, n=None):
        k = len(counts)
        return lib.wtconv_grad_norm(k if n is None else n, (ctypes.c_void_p * k)(*grads), (ctypes.c_int64 * k)(*counts),
                                    (ctypes.c_int32 * k)(*dtypes), max_norm, step, out, ws, bytes_, None)

    for kw, status in ((dict(n=-1), 1), (dict(out=None), 1), (dict(out=(3 << 40) + 2), 1), (dict(max_norm=0.0), 1),
                       (dict(max_norm=float("nan")), 1), (dict(max_norm=-1.0), 1), (dict(dtypes=(0, 2)), 1),
                       (dict(grads=((1 << 40) + 2, 2 << 40)), 1), (dict(grads=(1 << 40, (2 << 40) + 1)), 1),
                       (dict(step=(5 << 40) + 4), 1), (dict(counts=(-1, 5)), 2), (dict(counts=(1, (1 << 34) + 1)), 2),
                       (dict(ws=None), 3), (dict(bytes_=need - 1), 3), (dict(ws=(4 << 40) + 4), 3), (dict(out=1 << 40), 1),
                       (dict(step=1 << 40), 1), (dict(ws=1 << 40), 1), (dict(grads=(1 << 48, 2 << 40)), 1), (dict(step=3 << 40), 1), (dict(out=(4 << 40) + 8), 1)):
        assert norm(**kw) == status, kw
    assert lib.wtconv_grad_norm(1, None, None, None, 1.0, None, P[0], P[1], 1 << 20, None) == 1


def test_optimizer_arguments():
    w = torch.nn.Parameter(torch.zeros(4))
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(betas=(1.0, 0.9)), dict(eps=0.0), dict(weight_decay=-0.1),
               dict(state_bits=16), dict(max_norm=0.0), dict(rng=torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            op.AdamW([w], **kw)
    with pytest.raises(ValueError):
        op.AdamW([w, torch.nn.Parameter(torch.zeros(4, dtype=torch.bfloat16))])
    with pytest.raises(ValueError):
        op.AdamW([torch.nn.Parameter(torch.zeros(4, dtype=torch.float16))])
    o = op.AdamW([dict(params=[w], lr=0.1), dict(params=[torch.nn.Parameter(torch.zeros(3, dtype=torch.bfloat16))])])
    assert [g["lr"] for g in o.param_groups] == [0.1, 1e-3]
    assert o.step() is None   # no gradients: nothing to do
    w.grad = torch.zeros(4)
    with pytest.raises((ValueError, RuntimeError)):
        o.step()   # not on the GPU


def test_optimizer_groups_without_parameters():
    w = torch.nn.Parameter(torch.zeros(4))
    for groups in ([[w], []], [[], [w]], [[]]):
        o = op.AdamW([dict(params=g) for g in groups])
        assert o.step() is None
        o.load_state_dict(o.state_dict())
    with pytest.raises(ValueError):
        op.AdamW([dict(params=[]), dict(params=[w]), dict(params=[torch.nn.Parameter(torch.zeros(4, device="meta"))])])


def test_optimizer_takes_contiguous_parameters():
    w = torch.zeros(4, 3, 2, 2).to(memory_format=torch.channels_last)
    with pytest.raises(ValueError, match="contiguous"):
        op.AdamW([torch.nn.Parameter(w)])
    op.AdamW([torch.nn.Parameter(w[:, :, :1, :1].contiguous())])


def _made(shapes, dtype=torch.float32, **kw):
    """An optimizer whose states are there (on the host: no step is taken)."""
    o = op.AdamW([torch.nn.Parameter(torch.randn(s).to(dtype)) for s in shapes], **kw)
    o._buffers, o._step = [o._make(g) for g in o.param_groups], torch.full((1,), 3)
    for t in o._buffers[0].values():
        t.copy_(torch.rand(t.shape))
    return o


@pytest.mark.parametrize("dtype,bits", [(torch.float32, 32), (torch.float32, 8), (torch.bfloat16, 32)])
@pytest.mark.parametrize("mine,theirs", [(((256,), (10,)), ((10,), (256,))), (((300, 2), (700,)), ((700,), (300, 2))),
                                         (((16, 8),), ((8, 16),)), (((100,), (0,)), ((0,), (100,)))])
def test_a_state_of_other_shapes_is_refused(lib, mine, theirs, dtype, bits):
    """Buffers of the same size whose tensors stand elsewhere."""
    saved = _made(mine, dtype, state_bits=bits).state_dict()
    for o in (_made(theirs, dtype, state_bits=bits),
              op.AdamW([torch.nn.Parameter(torch.zeros(s, dtype=dtype)) for s in theirs], state_bits=bits)):
        before = [None if b is None else {k: t.clone() for k, t in b.items()} for b in o._buffers], o._step
        with pytest.raises(ValueError, match="other parameters"):
            o.load_state_dict(saved)
        assert o._step is before[1]
        assert all(b is a or all(torch.equal(a[k].float(), b[k].float()) for k in a) for a, b in zip(before[0], o._buffers))
    same = _made(mine, dtype, state_bits=bits)
    same.load_state_dict(saved)
    assert all(torch.equal(same._buffers[0][k].float(), t.float()) for k, t in saved["state"]["buffers"][0].items())


def test_a_state_without_shapes_is_loaded(lib):
    """As states were saved that did not hold them."""
    saved = _made(((7, 3), (300,))).state_dict()
    del saved["state"]["shapes"]
    o = _made(((7, 3), (300,)))
    o.load_state_dict(saved)
    assert all(torch.equal(o._buffers[0][k], t) for k, t in saved["state"]["buffers"][0].items())


def test_a_state_without_buffers_is_loaded_for_any_shapes():
    """There is nothing in it that belongs to a parameter."""
    saved = op.AdamW([torch.nn.Parameter(torch.zeros(4, 2))], lr=0.5).state_dict()
    o = op.AdamW([torch.nn.Parameter(torch.zeros(9))])
    o.load_state_dict(saved)
    assert o.param_groups[0]["lr"] == 0.5 and o._buffers == [None]


@pytest.mark.parametrize("kw,status", [*test_bad_steps.pytestmark[0].args[1], (dict(), 0), (dict(counts=(0, 0)), 0),
                                       (dict(state_bits=8, scales=8 << 40, rng=9 << 40, site=(1 << 31) - 2), 0),
                                       (dict(p_dtype=1, master=8 << 40), 0), (dict(grads=(None, None)), 0)])
def test_the_check_of_a_step_says_what_the_step_says(lib, kw, status, monkeypatch):
    """Where it finds nothing, too: nothing is launched."""
    class Check:
        wtconv_adamw_step = staticmethod(lambda *a: lib.wtconv_adamw_check(*a[:-1]))
    assert _adamw(Check, **kw) == status


def test_optimizer_numbers():
    """What a step would refuse is refused when the group is added, and a refused group is not there afterwards."""
    w, b = torch.nn.Parameter(torch.zeros(4)), torch.nn.Parameter(torch.zeros(3))
    good = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
    bad = [dict(eps=1e-40), dict(eps=float("inf")), dict(eps=1e39), dict(eps=float("nan")), dict(lr=1e39), dict(lr="fast"),
           dict(lr=None), dict(lr=torch.ones(2)), dict(weight_decay=float("nan")), dict(weight_decay=1e39),
           dict(betas=0.9), dict(betas=(0.9,)), dict(betas=(0.9, 0.99, 0.999)), dict(betas=("a", "b")),
           dict(betas=(0.9, float("nan"))), dict(eps=None), dict(weight_decay=[0.1])]
    for kw in bad:
        with pytest.raises(ValueError):
            op.AdamW([w], **{**good, **kw})
        o = op.AdamW([w], **good)
        with pytest.raises(ValueError):
            o.add_param_group({"params": [b], **good, **kw})
        assert len(o.param_groups) == len(o._buffers) == 1
    for kw in (dict(eps=1.18e-38), dict(eps=torch.tensor(1e-6)), dict(lr=torch.tensor(1e-3)), dict(lr=0), dict(betas=[0.0, 0.5]),
               dict(lr=torch.tensor([1e-3], dtype=torch.float64)), dict(weight_decay=0)):
        o = op.AdamW([w], **{**good, **kw})
        o.add_param_group({"params": [b]})
        assert len(o.param_groups) == len(o._buffers) == 2
    with pytest.raises(ValueError, match="lr_factor"):   # a rate that is not on the host
        op.AdamW([w], lr=torch.ones((), device="meta"))


def test_the_optimizer_s_sites_are_not_the_dropouts():
    """One rng serves a whole model, whose dropouts are numbered from 0 on; sites are below 2^31."""
    w = [torch.nn.Parameter(torch.zeros(4)) for _ in range(3)]
    assert op.AdamW(w).site == op.AdamW(w, state_bits=8, rng=torch.zeros(2, dtype=torch.int64)).site == 1 << 30
    assert op.AdamW(w, site=7).site == 7
