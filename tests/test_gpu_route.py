"""The router's choice, the grouping of rows and the weighted sum against plain implementations in 64 bits.

Tolerances: route, the steps that groups_ref counts; combine, one rounding of 2^-24 of the sum of the terms'
magnitudes a slot and one for the residual, and half a step of the output's type.  The rest is equal.
"""
import numpy as np
import pytest

import groups_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_02_amd as m

    m.lib()
    return m


def check_route(bqm, x, top, renorm):
    m = x.shape[0]
    ids = torch.full((m, top), 77, dtype=torch.int32, device=DEV)
    w = torch.full((m, top), 77.0, device=DEV)
    bqm.bqm_route(x, top, renorm, ids=ids, weights=w)
    want_ids, want, steps = groups_ref.route(x.cpu().double().numpy(), top, renorm)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = w.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    # weights below the smallest normal f32 keep fewer bits
    err, tol = np.abs(got - want), np.maximum(steps * 2.0 ** -24 * want, 2.0 ** -148)
    assert (np.nan_to_num(err) <= np.nan_to_num(tol)).all(), np.nanmax(err / tol)


@pytest.mark.parametrize("e,top", [(1, 1), (2, 2), (3, 1), (8, 2), (63, 4), (64, 8), (65, 8), (128, 8), (200, 32),
                                   (256, 8), (257, 6), (511, 10), (512, 32), (777, 1), (1023, 8), (1024, 32)])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("renorm", [True, False])
def test_route_random(bqm, e, top, t, renorm):
    g = torch.Generator().manual_seed(e * 100 + top)
    for m in (1, 5, 130):
        check_route(bqm, (torch.randn((m, e), generator=g) * 2.5).to(t).to(DEV), top, renorm)


@pytest.mark.parametrize("e", [5, 64, 200, 1024])
def test_route_ties_go_to_the_lowest_column(bqm, e):
    g = torch.Generator().manual_seed(e)
    x = torch.randint(-2, 3, (64, e), generator=g).float()
    x[0] = 1.0
    x[1] = torch.where(torch.arange(e) % 2 == 0, 0.0, -0.0)
    x[2] = torch.where(torch.arange(e) % 2 == 0, -0.0, 0.0)
    check_route(bqm, x.to(DEV), min(e, 32), True)


@pytest.mark.parametrize("e", [6, 64, 130, 1000])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_masks_infinities_and_nan(bqm, e, renorm):
    g = torch.Generator().manual_seed(e)
    x = torch.randn((12, e), generator=g)
    x[0] = -float("inf")                                    # nothing is left
    x[1, 1:] = -float("inf")                                # one is left, the first
    x[2, :-1] = -float("inf")                               # the last
    x[3, torch.randperm(e, generator=g)[: e - 4]] = -float("inf")
    x[4, 2] = float("nan")
    x[5] = float("nan")
    x[6, 3] = float("inf")
    x[7, 3] = x[7, 1] = float("inf")
    x[8] = torch.finfo(torch.float32).min                   # masked with the type's lowest value: still numbers
    x[9, 1:] = torch.finfo(torch.float32).min
    x[10] = 3e38
    x[10, 0] = -3e38                                        # the difference overflows to -inf: weight 0
    x[11, 0], x[11, 1] = float("nan"), float("-inf")
    check_route(bqm, x.to(DEV), 6, renorm)


def test_route_strided_rows(bqm):
    wide = torch.randn((9, 300), generator=torch.Generator().manual_seed(1)).to(DEV)
    for t in TYPES:
        check_route(bqm, wide.to(t)[:, 3:3 + 129], 8, True)
        check_route(bqm, wide.to(t)[::2, 1:65], 4, False)


@pytest.mark.parametrize("count", [1, 2, 63, 64, 65, 1000, 4095, 4096, 4097, 8192, 20001, 70000])
@pytest.mark.parametrize("groups", [1, 2, 7, 64, 255, 256, 1023, 1024])
def test_group_rows(bqm, count, groups):
    rng = np.random.default_rng(count + groups)
    ids = rng.integers(-1, groups + 1, count)
    ids[rng.random(count) < 0.3] = groups // 2
    check_groups(bqm, ids, groups)


def check_groups(bqm, ids, groups):
    count = len(ids)
    offsets = torch.full((groups + 1,), -7, dtype=torch.int32, device=DEV)
    order = torch.full((count,), -7, dtype=torch.int32, device=DEV)
    need = bqm.bqm_group_rows_workspace(count, groups)
    guard = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    bqm.bqm_group_rows(torch.from_numpy(ids.astype(np.int32)).to(DEV), groups, offsets, order, guard)
    want_offsets, want_order = groups_ref.group_rows(ids, groups)
    assert np.array_equal(offsets.cpu().numpy(), want_offsets) and np.array_equal(order.cpu().numpy(), want_order)
    assert bool((guard[need:] == 0x5A).all())


@pytest.mark.parametrize("count", [1, 100, 4096, 9000])
def test_group_rows_of_one_group_of_none_and_out_of_range(bqm, count):
    lowest, most = -2 ** 31, 2 ** 31 - 1
    check_groups(bqm, np.full(count, 3), 8)
    check_groups(bqm, np.full(count, 7), 8)
    check_groups(bqm, np.full(count, -1), 8)
    check_groups(bqm, np.full(count, 1023), 1024)
    check_groups(bqm, np.random.default_rng(1).choice([lowest, -1, 0, 1, 7, 8, 9, 1 << 20, most], count), 8)


def test_group_rows_many(bqm):
    """Over two million rows: 512 chunks."""
    ids = np.random.default_rng(3).integers(-1, 130, 2_097_155)
    check_groups(bqm, ids, 128)


def test_group_rows_the_most(bqm):
    rng = np.random.default_rng(4)
    check_groups(bqm, rng.integers(-1, 1025, bqm.MAX_ROWS).astype(np.int16), 1024)


@pytest.mark.parametrize("count", [1, 7, 63, 64, 65])
@pytest.mark.parametrize("groups", [1, 63, 64, 65, 255, 256, 257])
def test_group_rows_few(bqm, count, groups):
    for seed in range(3):
        check_groups(bqm, np.random.default_rng(seed).integers(-1, groups + 1, count), groups)


def combine_ref(y, w, res, m, top):
    v = y.cpu().double().numpy().reshape(m, top, -1)
    c = w.cpu().double().numpy()[:, :, None]
    with np.errstate(invalid="ignore"):
        terms = np.where(c != 0, c * v, 0.0)
    out, total = terms.sum(1), np.abs(terms).sum(1)
    if res is not None:
        out, total = out + res.cpu().double().numpy(), total + np.abs(res.cpu().double().numpy())
    return out, total


@pytest.mark.parametrize("m,top,n", [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (5, 6, 129), (7, 9, 520), (33, 32, 264), (2, 10, 5121)])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("with_res", [False, True])
def test_combine(bqm, m, top, n, t, same, with_res):
    g = torch.Generator().manual_seed(m + n)
    y = torch.randn((m * top, n), generator=g).to(t).to(DEV)
    w = torch.rand((m, top), generator=g).to(DEV)
    ot = t if same else torch.float32
    res = (4 * torch.randn((m, n), generator=g)).to(ot).to(DEV) if with_res else None
    out = torch.full((m, n), 77.0, dtype=ot, device=DEV)
    bqm.bqm_combine(y, w, res, out=out)
    want, total = combine_ref(y, w, res, m, top)
    sums = (top + 1) * 2.0 ** -24 * total
    eps = torch.finfo(ot).eps
    tol = sums + (0 if ot == torch.float32 else groups_ref.half_step(np.abs(want) + sums, eps, 2.0 ** -24 if ot == torch.float16 else 2.0 ** -133))
    assert (np.abs(out.cpu().double().numpy() - want) <= tol).all()
    if with_res:                                             # in place
        assert bqm.bqm_combine(y, w, res, out=res) is res and torch.equal(res, out)


def test_combine_weight_zero_adds_nothing(bqm):
    y = torch.ones((6, 40), device=DEV)
    y[1], y[4] = float("nan"), float("inf")
    w = torch.tensor([[1.0, 0.0, 2.0], [0.5, -0.0, 0.0]], device=DEV)
    out = bqm.bqm_combine(y, w)
    assert bool((out[0] == 3).all()) and bool((out[1] == 0.5).all())


def test_combine_nan_where_the_formula_has_it(bqm):
    y = torch.ones((4, 9), device=DEV)
    y[3, 2] = float("inf")
    w = torch.tensor([[float("nan"), 1.0], [1.0, 1.0]], device=DEV)
    out = bqm.bqm_combine(y, w).cpu()
    assert bool(out[0].isnan().all()) and out[1, 2] == float("inf") and out[1, 1] == 2


def test_combine_unaligned_rows(bqm):
    flat = torch.randn(8 * 64 + 1, generator=torch.Generator().manual_seed(2)).to(DEV)
    w = torch.rand((4, 2), generator=torch.Generator().manual_seed(3)).to(DEV)
    a, b = flat[1:].view(8, 64), flat[1:].clone().view(8, 64)
    assert torch.equal(bqm.bqm_combine(a, w), bqm.bqm_combine(b, w))


@pytest.mark.parametrize("top", [1, 3, 9])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("same", [False, True])
def test_combine_ragged_rows_in_place(bqm, top, t, same):
    """Rows of every rest of 16 bytes, from bases that are aligned to an element only, in place and not, and what lies
    on either side of out."""
    m, ot = 5, t if same else torch.float32
    for n in list(range(1, 26)) + [1029, 2055]:
        g = torch.Generator().manual_seed(n)
        y = torch.randn(m * top * n + 1, generator=g).to(t).to(DEV)[1:].view(m * top, n)
        w = torch.rand((m, top), generator=g).to(DEV)
        res = torch.randn((m, n), generator=g).to(ot).to(DEV)
        flat = torch.full((m * n + 16,), 77.0, dtype=ot, device=DEV)
        out = flat[1:1 + m * n].view(m, n)
        bqm.bqm_combine(y, w, res, out=out)
        want, total = combine_ref(y, w, res, m, top)
        sums = (top + 1) * 2.0 ** -24 * total                # a rounding of 2^-24 of the terms' sum each
        tol = sums + (0 if ot == torch.float32 else groups_ref.half_step(np.abs(want) + sums, torch.finfo(ot).eps, 2.0 ** -24 if ot == torch.float16 else 2.0 ** -133))
        assert (np.abs(out.cpu().double().numpy() - want) <= tol).all(), n
        assert bool((flat[:1] == 77).all()) and bool((flat[1 + m * n:] == 77).all()), n
        kept = out.clone()
        out.copy_(res)
        assert bqm.bqm_combine(y, w, out, out=out) is out and torch.equal(out, kept), n
        assert bool((flat[:1] == 77).all()) and bool((flat[1 + m * n:] == 77).all()), n
