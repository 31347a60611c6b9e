"""Expert rows: slots sorted by expert, rows there and back, and their
gradients, against plain forms in 64 bits (tests/_step_ref.py)."""
import pytest
import torch

from tests._step_ref import live_of, rows_ref, sort_ref, sum_bwd_ref, sum_ref
from wavelet_convolution_amd import expert_binding as eb
from wavelet_convolution_amd import experts as ex

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16]


def ids(N, K, E, seed=0, dropped=0.1, dtype=torch.int64, skew=True):
    """Experts of [N, K] slots, some of them none (numbers on either side of the range)."""
    g = torch.Generator().manual_seed(seed)
    e = (torch.rand(N, K, generator=g) ** (2 if skew else 1) * E).long().clamp(max=E - 1)
    out = torch.rand(N, K, generator=g) < dropped
    e[out] = torch.where(torch.rand(int(out.sum()), generator=g) < 0.5, -1 - e[out], E + e[out])
    return e.to(DEV, dtype)


def same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a.cpu().long(), torch.as_tensor(b).long())


# sizes around a group of 64, one workgroup's share and the parts of several
SORTS = [(1, 1, 1), (1, 2, 8), (63, 1, 3), (64, 2, 2), (65, 1, 1), (7, 5, 1024), (1000, 3, 5), (4096, 2, 16),
         (4097, 2, 16), (8193, 1, 1), (9000, 1, 1000), (20000, 8, 256), (50000, 2, 64), (100_352, 4, 511),
         (300_001, 2, 512), (1_200_007, 1, 7)]


@pytest.mark.parametrize("N,K,E", SORTS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(N, K, E, dtype):
    e = ids(N, K, E, dtype=dtype)
    got = eb.wtconv_expert_sort(e, E)
    same(got, sort_ref(e, E))
    assert all(t.dtype == torch.int32 for t in got) and got[1].shape == e.shape
    again = eb.wtconv_expert_sort(e, E)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


# on both sides of where parts change their size, and counts the way they are summed up
@pytest.mark.parametrize("N,K,E", [(2048, 2, 63), (2048, 2, 64), (4096, 1, 1023), (4097, 1, 16), (16_385, 1, 255),
                                   (24_577, 1, 256), (262_144, 1, 16), (262_145, 1, 16), (131_072, 2, 128),
                                   (131_073, 2, 128), (65_537, 1, 1024), (1_048_576, 1, 32), (1_048_577, 1, 16),
                                   (2_097_153, 1, 3), (2_500_000, 1, 1024), (8_388_608, 2, 5), (8_388_609, 2, 5)])
def test_sort_in_parts(N, K, E):
    e = ids(N, K, E, dtype=torch.int32)
    same(eb.wtconv_expert_sort(e, E), sort_ref(e, E))


def check_stable(e, E, got):
    """order, place and offsets are those of a stable sort, by what defines them: places and slots undo each other,
    experts do not fall along the places, the slots of one rise, and offsets count. In pieces, for many slots."""
    order, place, offsets = got
    order, flat, place, S = order.view(-1), e.reshape(-1), place.view(-1), e.numel()
    count, last = torch.zeros(E + 1, dtype=torch.int64, device=DEV), (-1, -1)
    for at in range(0, S, 1 << 27):
        slots = order[at:at + (1 << 27)].long()
        assert int(slots.min()) >= 0 and int(slots.max()) < S, at
        assert torch.equal(place[slots].long(), torch.arange(at, at + len(slots), device=DEV)), at
        key = flat[slots].long()
        key = torch.where((key < 0) | (key >= E), E, key)
        assert (int(key[0]), int(slots[0])) > last, at
        assert ((key[1:] > key[:-1]) | ((key[1:] == key[:-1]) & (slots[1:] > slots[:-1]))).all(), at
        count += torch.bincount(key, minlength=E + 1)
        last = int(key[-1]), int(slots[-1])
    assert torch.equal(offsets[1:].long(), count.cumsum(0)[:E]) and int(offsets[0]) == 0


@pytest.mark.parametrize("E", [1, 2, 3, 4, 64])
@pytest.mark.parametrize("S", [2 ** 24, 2 ** 24 + 1, 100_000_003])
def test_sort_of_more_slots_than_the_parts_hold(S, E):
    """From 2^24 slots on a part has more slots than a workgroup's wavefronts hold in registers."""
    g = torch.Generator(DEV).manual_seed(S + E)
    e = torch.randint(-1 if E > 1 else 0, E + 1, (S, 1), generator=g, device=DEV, dtype=torch.int32)
    check_stable(e, E, eb.wtconv_expert_sort(e, E))


@pytest.mark.parametrize("E", [3, 1000])
def test_sort_of_as_many_slots_as_there_are_places(E):
    S = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 64 * 2 ** 30:
        pytest.skip("needs 64 GiB")
    e = torch.empty(S, 1, device=DEV, dtype=torch.int32).random_(0, E + 1, generator=torch.Generator(DEV).manual_seed(E))
    check_stable(e, E, eb.wtconv_expert_sort(e, E))


def test_stable_sorts_are_told_from_others():
    e = ids(5000, 2, 7)
    order, place, offsets = eb.wtconv_expert_sort(e, 7)
    check_stable(e, 7, (order, place, offsets))
    other = order.clone()
    other[:2] = order[:2].flip(0)   # two slots of one expert
    turned = torch.empty_like(place.view(-1))
    turned[other.long()] = torch.arange(len(other), device=DEV, dtype=torch.int32)
    for bad in ((other, turned, offsets), (order, turned, offsets), (other, place, offsets), (order, place, offsets + 1)):
        with pytest.raises(AssertionError):
            check_stable(e, 7, bad)


@pytest.mark.parametrize("N", [1, 700, 9000])
@pytest.mark.parametrize("what", ["one", "last", "none", "far", "in order", "backwards"])
def test_sort_of_extremes(N, what):
    K, E = 2, 33
    e = {"one": torch.zeros(N, K), "last": torch.full((N, K), E - 1), "none": torch.full((N, K), -1),
         "far": torch.full((N, K), 2 ** 40 + 3, dtype=torch.int64),
         "in order": torch.arange(N * K).view(N, K) * E // (N * K),
         "backwards": (N * K - 1 - torch.arange(N * K)).view(N, K) * E // (N * K)}[what].to(DEV, torch.int64)
    same(eb.wtconv_expert_sort(e, E), sort_ref(e, E))


def test_sort_of_nothing():
    order, place, offsets = eb.wtconv_expert_sort(torch.empty(0, 3, dtype=torch.int64, device=DEV), 5)
    assert order.shape == (0,) and place.shape == (0, 3) and offsets.tolist() == [0] * 6


def test_sort_into_given_tensors():
    e = ids(20_000, 2, 16)
    n = e.numel()
    out = dict(order=torch.full((n,), -7, dtype=torch.int32, device=DEV), place=torch.empty_like(e, dtype=torch.int32),
               offsets=torch.empty(17, dtype=torch.int32, device=DEV))
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)   # what stands there does not count
    got = eb.wtconv_expert_sort(e, 16, ws=ws, **out)
    assert all(a is b for a, b in zip(got, out.values()))
    same(got, sort_ref(e, 16))


# channels around the vector of eight, the lanes of a row and odd widths
WIDTHS = [1, 3, 7, 8, 9, 12, 31, 96, 97, 100, 192, 384, 513, 1024, 1536, 2050]


def routed(N, K, E, C, t, seed=0, dropped=0.1):
    e = ids(N, K, E, seed, dropped)
    order, place, offsets = eb.wtconv_expert_sort(e, E)
    g = torch.Generator(DEV).manual_seed(seed + 1)
    x, dy = (torch.randn(N, C, generator=g, device=DEV).to(t) for _ in range(2))
    ys = torch.randn(N * K, C, generator=g, device=DEV).to(t)
    w = torch.rand(N, K, generator=g, device=DEV)
    # nothing of a slot without an expert is looked at
    dead = ~live_of(place, offsets)
    ys[place.view(-1).long()[dead]] = float("nan")
    w.view(-1)[dead] = float("nan")
    return place, offsets, x, ys, w, dy


def near(got, want, bound):
    off = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all()
    assert (off <= bound).all(), float((off / bound).max())


def check_all(place, offsets, x, ys, w, dy):
    xs = eb.wtconv_expert_rows_fwd(x, place, offsets)
    assert torch.equal(xs, rows_ref(x, place, offsets)[0])
    near(eb.wtconv_expert_rows_bwd(ys, place, offsets), *sum_ref(ys, None, place, offsets))
    near(eb.wtconv_expert_sum_fwd(ys, w, place, offsets), *sum_ref(ys, w, place, offsets))
    dys, dw = eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets)
    want = sum_bwd_ref(dy, ys, w, place, offsets)
    near(dys, *want[0])
    near(dw, *want[1])
    only = eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets, want=["dys"])
    assert only[1] is None and torch.equal(only[0], dys)
    only = eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets, want=["dweight"])
    assert only[0] is None and torch.equal(only[1], dw)
    assert eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets, want=()) == (None, None)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_rows_of_any_width(C, t):
    check_all(*routed(131, 2, 5, C, t))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("N,K,E,C", [(1, 1, 1, 8), (1, 2, 8, 384), (1, 8, 256, 1536), (5, 3, 4, 97), (257, 4, 9, 40),
                                     (33, 5, 7, 100), (1000, 1, 64, 96), (77, 8, 8, 24), (3, 70, 2, 16),
                                     (2047, 2, 64, 1024), (12_544, 2, 16, 192)])
def test_rows_of_any_number(N, K, E, C, t):
    check_all(*routed(N, K, E, C, t, seed=3))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dropped", [0.0, 1.0])
def test_all_or_no_slots_have_an_expert(t, dropped):
    place, offsets, x, ys, w, dy = routed(300, 2, 4, 48, t, dropped=dropped)
    check_all(place, offsets, x, ys, w, dy)
    if dropped == 1.0:
        assert int(offsets[-1]) == 0
        assert not eb.wtconv_expert_sum_fwd(ys, w, place, offsets).any()


def test_places_that_are_none():
    """A place out of range counts as none; a row of xs or dys that no place names stays as it is."""
    place, offsets, x, ys, w, dy = routed(200, 2, 4, 40, torch.float32, dropped=0.0)
    place = place.clone()
    place[3, 0], place[7, 1], place[9] = -1, 400, torch.tensor([2 ** 31 - 1, -2 ** 31], device=DEV, dtype=torch.int32)
    xs = torch.full_like(ys, 5.0)
    eb.wtconv_expert_rows_fwd(x, place, offsets, xs=xs)
    want, written = rows_ref(x, place, offsets)
    assert torch.equal(xs[written], want[written]) and (xs[~written] == 5).all() and int((~written).sum()) == 4
    near(eb.wtconv_expert_rows_bwd(ys, place, offsets), *sum_ref(ys, None, place, offsets))
    near(eb.wtconv_expert_sum_fwd(ys, w, place, offsets), *sum_ref(ys, w, place, offsets))
    dys, dw = eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets)
    (want, bound), wants = sum_bwd_ref(dy, ys, w, place, offsets)
    near(dys[written], want[written], bound[written])
    near(dw, *wants)


def test_no_rows():
    place = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    offsets = torch.zeros(4, dtype=torch.int32, device=DEV)
    x, w = torch.empty(0, 16, device=DEV), torch.empty(0, 2, device=DEV)
    assert eb.wtconv_expert_rows_fwd(x, place, offsets).shape == (0, 16)
    assert eb.wtconv_expert_rows_bwd(x, place, offsets).shape == (0, 16)
    assert eb.wtconv_expert_sum_fwd(x, w, place, offsets).shape == (0, 16)
    assert [t.shape for t in eb.wtconv_expert_sum_bwd(x, x, w, place, offsets)] == [(0, 16), (0, 2)]


def test_infinities_and_nan_stay_in_their_rows():
    place, offsets, x, ys, w, dy = routed(64, 2, 4, 24, torch.bfloat16, dropped=0.0)
    x[5, 3], x[6, 1] = float("inf"), float("nan")
    xs = eb.wtconv_expert_rows_fwd(x, place, offsets)
    assert torch.equal(xs.isnan().any(1).nonzero().view(-1).int(), place[6].sort().values)
    assert torch.equal(xs.isinf().any(1).nonzero().view(-1).int(), place[5].sort().values)
    ys[place[9, 1].long(), 2] = float("inf")
    y = eb.wtconv_expert_sum_fwd(ys, w, place, offsets)
    assert y.isinf().nonzero().tolist() == [[9, 2]] and not y.isnan().any()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("C", [5, 8, 21, 97, 200])
def test_infinities_do_not_reach_other_sums(C, t):
    """An infinity in dy or ys gives infinite products in its own slots, none in slots without an expert, and no NaN
    where a row's vectors overlap."""
    N, K, E = 70, 2, 4
    place, offsets, x, ys, w, dy = routed(N, K, E, C, t)
    live = live_of(place, offsets).view(N, K)
    ys[torch.arange(N * K, device=DEV) < offsets[-1]] = 1
    dy.fill_(1)
    one = int(live.all(1).nonzero()[0])
    for j in range(C):
        for row in (0, one, int((~live).any(1).nonzero()[0])):
            bad = dy.clone()
            bad[row, j] = float("inf")
            dys, dw = eb.wtconv_expert_sum_bwd(bad, ys, w, place, offsets)
            want = torch.where(live, float(C), 0.0)
            want[row] = torch.where(live[row], float("inf"), 0.0)
            assert torch.equal(dw, want), (C, j, row)
        bad = ys.clone()
        bad[place[one, 0].long(), j] = float("inf")
        want = torch.where(live, float(C), 0.0)
        want[one, 0] = float("inf")
        assert torch.equal(eb.wtconv_expert_sum_bwd(dy, bad, w, place, offsets)[1], want), (C, j)


@pytest.mark.parametrize("t", TYPES)
def test_pointers_aligned_to_the_element_only(t):
    place, offsets, x, ys, w, dy = routed(90, 2, 4, 33, t)

    def moved(a):
        b = torch.empty(a.numel() + 1, dtype=a.dtype, device=DEV)[1:].view(a.shape)
        return b.copy_(a)

    check_all(moved(place), moved(offsets), moved(x), moved(ys), moved(w), moved(dy))


def test_more_elements_than_32_bits_count():
    """2^21 slots of 2,056 channels: the last rows of more than 2^32 elements."""
    N, K, C = 1 << 20, 2, 2056
    place = torch.arange(N * K - 1, -1, -1, dtype=torch.int32, device=DEV).view(N, K)   # backwards
    offsets = torch.tensor([0, N * K], dtype=torch.int32, device=DEV)
    x = torch.arange(N, device=DEV).remainder(251).to(torch.bfloat16).view(N, 1).expand(N, C).contiguous()
    xs = eb.wtconv_expert_rows_fwd(x, place, offsets)
    want = torch.arange(N * K - 1, -1, -1, device=DEV).div(2, rounding_mode="floor").remainder(251).to(torch.bfloat16)
    for c in (0, 1000, C - 1):
        assert torch.equal(xs[:, c], want)
    w = torch.tensor([0.25, 0.5], device=DEV).expand(N, K).contiguous()
    y = eb.wtconv_expert_sum_fwd(xs, w, place, offsets)
    for c in (0, 1000, C - 1):
        assert torch.equal(y[:, c], (x[:, c].float() * 0.75).to(torch.bfloat16))
    dys, dw = eb.wtconv_expert_sum_bwd(x, xs, w, place, offsets)
    each = (x[:, :1].float() * w).to(torch.bfloat16).view(-1).flip(0)
    for c in (0, 1000, C - 1):
        assert torch.equal(dys[:, c], each)
    assert torch.equal(dw[:, 0], dw[:, 1]) and torch.equal(dw[:, 0], x[:, 0].float() ** 2 * C)   # whole numbers


# ---------------------------------------------------------------- autograd

def test_gradients_through_autograd():
    """Leading dimensions, sums of other losses, and the formula's gradients (the plain form's, differentiated)."""
    B, H, W, K, E, C = 2, 3, 5, 2, 4, 20
    e = ids(B * H * W, K, E).view(B, H, W, K)
    route = ex.expert_sort(e, E)
    g = torch.Generator(DEV).manual_seed(5)
    x = torch.randn(B, H, W, C, generator=g, device=DEV, requires_grad=True)
    w = torch.rand(B, H, W, K, generator=g, device=DEV, requires_grad=True)
    dy = torch.randn(B, H, W, C, generator=g, device=DEV)
    y = ex.expert_sum(torch.tanh(ex.expert_rows(x, route)), w, route)
    assert y.shape == x.shape
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    xd, wd = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    live = live_of(route.place, route.offsets).view(e.shape).double()
    yd = (torch.tanh(xd).unsqueeze(3) * (wd * live).unsqueeze(-1)).sum(3)
    want = torch.autograd.grad(yd, (xd, wd), dy.double())
    # tanh's own error in fp32 (a few steps) beside the rounded sums
    for a, b in ((y, yd), (dx, want[0]), (dw, want[1])):
        assert (a.double() - b).abs().max() <= 2e-5 * b.abs().max()


def test_any_memory_order_through_autograd():
    """Planar activations, transposed weights and experts, an expanded gradient."""
    B, C, H, W, K, E = 2, 12, 3, 5, 2, 4
    e = ids(K, B * H * W, E, dropped=0.0).view(K, B, H, W).permute(1, 2, 3, 0)
    x = torch.randn(B, C, H, W, device=DEV, requires_grad=True)
    w = torch.rand(K, B, H, W, device=DEV, requires_grad=True)
    route = ex.expert_sort(e, E)
    y = ex.expert_sum(ex.expert_rows(x.permute(0, 2, 3, 1), route), w.permute(1, 2, 3, 0), route)
    dx, dw = torch.autograd.grad(y.sum(), (x, w))
    assert (dx - w.sum(0).unsqueeze(1)).abs().max() <= 1e-6
    assert (dw - x.sum(1).unsqueeze(0)).abs().max() <= C * 1e-6


def test_gradients_against_differences():
    """rows and sum are linear in each argument: central differences with powers of two are exact up to rounding."""
    place, offsets, x, ys, w, dy = routed(40, 3, 4, 12, torch.float32, dropped=0.0)
    h = 0.5
    dys, dw = eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets)
    for (i, j) in ((0, 0), (17, 5), (119, 11)):
        d = torch.zeros_like(ys)
        d[i, j] = h
        up, down = (eb.wtconv_expert_sum_fwd(ys + s * d, w, place, offsets).double() for s in (1, -1))
        slope = ((up - down) * dy.double()).sum() / (2 * h)
        assert abs(float(slope - dys[i, j])) <= 1e-5
    for (i, j) in ((0, 0), (21, 2)):
        d = torch.zeros_like(w)
        d[i, j] = h
        up, down = (eb.wtconv_expert_sum_fwd(ys, w + s * d, place, offsets).double() for s in (1, -1))
        slope = ((up - down) * dy.double()).sum() / (2 * h)
        assert abs(float(slope - dw[i, j])) <= 1e-5 * 12
    dxs = torch.randn_like(ys)
    dx = eb.wtconv_expert_rows_bwd(dxs, place, offsets)
    d = torch.zeros_like(x)
    d[7, 3] = h
    up, down = (eb.wtconv_expert_rows_fwd(x + s * d, place, offsets).double() for s in (1, -1))
    assert abs(float(((up - down) * dxs.double()).sum() / (2 * h) - dx[7, 3])) <= 1e-5


def test_only_wanted_gradients_and_no_second_one():
    route = ex.expert_sort(ids(30, 2, 4), 4)
    ys, w = torch.randn(60, 16, device=DEV), torch.rand(30, 2, device=DEV, requires_grad=True)
    y = ex.expert_sum(ys, w, route)
    dw, = torch.autograd.grad(y.sum(), w, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dw.sum(), w)


# -------------------------------------------------- streams, graphs, refusals

def test_on_another_stream():
    s = torch.cuda.Stream()
    e = ids(30_000, 2, 16)
    place, offsets, x, ys, w, dy = routed(500, 2, 4, 64, torch.bfloat16)
    torch.cuda.synchronize()
    got = eb.wtconv_expert_sort(e, 16, stream=s)
    xs = eb.wtconv_expert_rows_fwd(x, place, offsets, stream=s)
    y = eb.wtconv_expert_sum_fwd(ys, w, place, offsets, stream=s)
    s.synchronize()
    same(got, sort_ref(e, 16))
    assert torch.equal(xs, rows_ref(x, place, offsets)[0])
    near(y, *sum_ref(ys, w, place, offsets))


def test_calls_at_once():
    """Sorts (with workspaces of their own) and sums on two streams at the same time."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    es = [ids(200_000, 2, 16 + i, seed=i) for i in range(2)]
    sets = [routed(20_000, 2, 8, 96, torch.bfloat16, seed=i) for i in range(2)]
    want = [eb.wtconv_expert_sum_bwd(s[5], s[3], s[4], s[0], s[1]) for s in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, s in enumerate(streams):
            place, offsets, x, ys, w, dy = sets[i]
            got.append((i, eb.wtconv_expert_sort(es[i], 16 + i, stream=s),
                        eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets, stream=s)))
    torch.cuda.synchronize()
    first = [next(g[1] for g in got if g[0] == i) for i in range(2)]
    for i in range(2):
        same(first[i], sort_ref(es[i], 16 + i))
    for i, a, b in got:
        assert all(torch.equal(x, y) for x, y in zip(a, first[i]))
        # bit for bit, NaN of slots that are not read apart
        assert all(torch.equal(x.nan_to_num(), y.nan_to_num()) for x, y in zip(b, want[i]))


@pytest.mark.parametrize("N", [200, 6000])   # one workgroup, and parts with a workspace
def test_captured_and_replayed(N):
    """Sort, rows, products, sum and gradients in one graph, replayed on other ids, rows and weights."""
    K, E, C = 2, 8, 40
    e, w = ids(N, K, E), torch.rand(N, K, device=DEV)
    x, dy = torch.randn(N, C, device=DEV), torch.randn(N, C, device=DEV)

    def step():
        order, place, offsets = eb.wtconv_expert_sort(e, E)
        xs = eb.wtconv_expert_rows_fwd(x, place, offsets)
        y = eb.wtconv_expert_sum_fwd(xs, w, place, offsets)
        dys, dw = eb.wtconv_expert_sum_bwd(dy, xs, w, place, offsets)
        return order, place, offsets, xs, y, dys, dw, eb.wtconv_expert_rows_bwd(dys, place, offsets)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (11, 12, 13):
        e.copy_(ids(N, K, E, seed))
        w.copy_(torch.rand(N, K, device=DEV))
        x.copy_(torch.randn(N, C, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)
        same(held[:3], sort_ref(e, E))


def test_backward_captured():
    """Forward and backward through autograd in a graph."""
    N, K, E, C = 300, 2, 4, 32
    e = ids(N, K, E)
    x = torch.randn(N, C, device=DEV, requires_grad=True)
    w = torch.rand(N, K, device=DEV, requires_grad=True)
    dy = torch.randn(N, C, device=DEV)

    def step():
        route = ex.expert_sort(e, E)
        return torch.autograd.grad(ex.expert_sum(ex.expert_rows(x, route) * 2, w, route), (x, w), dy)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        dy.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_refusals_on_the_gpu():
    place, offsets, x, ys, w, dy = routed(20, 2, 4, 16, torch.float32)
    bad = [lambda: eb.wtconv_expert_sort(place.float(), 4), lambda: eb.wtconv_expert_sort(place[:, 0], 4),
           lambda: eb.wtconv_expert_sort(ids(20, 2, 4).t(), 4), lambda: eb.wtconv_expert_sort(place.cpu(), 4),
           lambda: eb.wtconv_expert_sort(place, 4, order=torch.empty(40, device=DEV)),
           lambda: eb.wtconv_expert_rows_fwd(x[:10], place, offsets), lambda: eb.wtconv_expert_rows_fwd(x.half(), place, offsets),
           lambda: eb.wtconv_expert_rows_fwd(x[:, ::2], place, offsets), lambda: eb.wtconv_expert_rows_fwd(x, place.long(), offsets),
           lambda: eb.wtconv_expert_rows_fwd(x, place, offsets.long()), lambda: eb.wtconv_expert_rows_fwd(x, place, offsets[:1]),
           lambda: eb.wtconv_expert_rows_fwd(x, place.cpu(), offsets),
           lambda: eb.wtconv_expert_rows_fwd(x, place, offsets, xs=ys.bfloat16()),
           lambda: eb.wtconv_expert_rows_bwd(x, place, offsets), lambda: eb.wtconv_expert_sum_fwd(ys, w.half(), place, offsets),
           lambda: eb.wtconv_expert_sum_fwd(ys, w[:, :1], place, offsets),
           lambda: eb.wtconv_expert_sum_bwd(dy.bfloat16(), ys, w, place, offsets),
           lambda: eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets, want=["dx"]),
           lambda: eb.wtconv_expert_sum_bwd(dy, x, w, place, offsets)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"case {i}")


def test_no_memory_is_torchs_error():
    """An output that does not fit raises what torch's own allocations raise."""
    x, place = torch.zeros(1 << 14, 512, device=DEV), torch.zeros(1 << 14, 64, dtype=torch.int32, device=DEV)
    offsets = torch.zeros(9, dtype=torch.int32, device=DEV)   # xs takes 2 GiB
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    try:
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + 2 ** 30) / total)
        with pytest.raises(torch.OutOfMemoryError):
            eb.wtconv_expert_rows_fwd(x, place, offsets)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert eb.wtconv_expert_rows_fwd(x[:16], place[:16], offsets).shape == (1024, 512)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("K", [1, 2, 5])
def test_what_a_sum_s_gradient_does_not_read_may_be_missing(K, t):
    place, offsets, x, ys, w, dy = routed(90, K, 4, 40, t)
    dys, dw = eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets)
    only = eb.wtconv_expert_sum_bwd(dy, None, w, place, offsets, want=["dys"])
    assert only[1] is None and torch.equal(only[0], dys)
    only = eb.wtconv_expert_sum_bwd(dy, ys, None, place, offsets, want=["dweight"])
    assert only[0] is None and torch.equal(only[1], dw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    only = eb.wtconv_expert_sum_bwd(dy, ys, None, place, offsets, want=["dweight"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(only[1], dw)
    assert eb.wtconv_expert_sum_bwd(dy, None, None, place, offsets, want=[]) == (None, None)
    for args, want in (((dy, None, w), ["dweight"]), ((dy, ys, None), ["dys"]), ((dy, None, w), ["dys", "dweight"]),
                       ((dy, ys, None), ["dys", "dweight"]), ((dy, ys[:1], w), ["dys"]), ((dy, ys, w[:1]), ["dweight"])):
        with pytest.raises(ValueError):
            eb.wtconv_expert_sum_bwd(*args, place, offsets, want=want)


def test_refusals_on_another_stream():
    """They are the same as on the current one."""
    place, offsets, x, ys, w, dy = routed(40, 2, 4, 16, torch.float32)
    e, s = ids(40, 2, 4), torch.cuda.Stream()
    for stream in (None, s):
        for call in (lambda: eb.wtconv_expert_sort(e, 4, place=place.cpu(), stream=stream),
                     lambda: eb.wtconv_expert_sort("e", 4, stream=stream),
                     lambda: eb.wtconv_expert_sort(e, 4, ws=[1], stream=stream),
                     lambda: eb.wtconv_expert_rows_fwd(x, place.cpu(), offsets, stream=stream),
                     lambda: eb.wtconv_expert_rows_fwd(None, place, offsets, stream=stream),
                     lambda: eb.wtconv_expert_rows_bwd(ys, place, offsets.cpu(), stream=stream),
                     lambda: eb.wtconv_expert_sum_fwd(ys, w.cpu(), place, offsets, stream=stream),
                     lambda: eb.wtconv_expert_sum_bwd(dy, ys.cpu(), w, place, offsets, stream=stream),
                     lambda: eb.wtconv_expert_sum_bwd(dy.cpu(), ys, w, place, offsets, stream=stream)):
            with pytest.raises(ValueError):
                call()


def test_given_outputs_are_seen_by_autograd():
    """A graph that needs what stood in a tensor before a call wrote it raises an error, as after torch's own
    operations in place."""
    e = ids(60, 2, 4)
    x = torch.randn(60, 16, device=DEV, requires_grad=True)
    w = torch.rand(60, 2, device=DEV)

    def graph():
        route = ex.expert_sort(e, 4)
        return route, ex.expert_sum(ex.expert_rows(x, route), w, route)

    for name in ("order", "place", "offsets"):
        route, y = graph()
        other = ids(60, 2, 4, seed=9)
        eb.wtconv_expert_sort(other, 4, **{name: getattr(route, name)})
        if name == "order":   # which no gradient needs
            y.sum().backward()
            continue
        with pytest.raises(RuntimeError, match="inplace"):
            y.sum().backward()
    place, offsets, rows, ys, w, dy = routed(30, 2, 4, 16, torch.float32)
    calls = {"xs": lambda t: eb.wtconv_expert_rows_fwd(rows, place, offsets, xs=t),
             "dx": lambda t: eb.wtconv_expert_rows_bwd(ys, place, offsets, dx=t),
             "y": lambda t: eb.wtconv_expert_sum_fwd(ys, w, place, offsets, y=t),
             "dys": lambda t: eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets, dys=t),
             "dweight": lambda t: eb.wtconv_expert_sum_bwd(dy, ys, w, place, offsets, dweight=t)}
    for name, call in calls.items():
        t = torch.empty_like({"xs": ys, "dys": ys, "dweight": w}.get(name, rows))
        before = t._version
        call(t)
        assert t._version == before + 1, name
        with torch.inference_mode():   # which keeps no record
            call(torch.empty_like(t))
    wrong = torch.empty(3, device=DEV)
    for call in calls.values():
        with pytest.raises(ValueError):
            call(wrong)
    assert wrong._version == 0
