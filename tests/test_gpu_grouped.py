"""The experts' products, grouped and for few slots, against 64 bits.

Tolerances, T = sum |terms|, on every output (as those of the products with one matrix):
* GEMM: a block's sum is exact, and each 64-k step adds two block sums to the accumulator, at most three cut or
  rounded additions of 2^-23: (3 k / 64 + 2) 2^-23 T.
* GEMV: exact products of the parts; a 32-k step sums 32 products and the accumulator, at most eight cut additions;
  16 steps for each 512 k of a wave, one in eight of the slices; then the waves and three parts:
  (8 * 16 * ceil(ceil(k / 512) / 8) + 8 + 4) 2^-23 T.
* With the gate, what groups_ref.gated makes of these; half a step of the output's type for 16-bit outputs.
"""
import numpy as np
import pytest

import groups_ref
import layer_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_02_amd as m

    m.lib()
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def random_mx(shape, k, rng, low=118, high=132):
    return (rng.integers(0, 256, (*shape, k // 2)).astype(np.uint8), rng.integers(low, high, (*shape, k // 32)).astype(np.uint8))


def plan(bqm, ids, groups):
    return bqm.bqm_group_rows(dev(ids.astype(np.int32)), groups)


def with_type(want, tol, t):
    if t == "f32":
        return tol
    eps = torch.finfo(TYPES[t]).eps
    return tol + groups_ref.half_step(np.abs(want) + tol, eps, 2.0 ** -24 if t == "f16" else 2.0 ** -133)


def gemm(bqm, w, ws, xq, xs, ids, glu, t="f32"):
    groups, n, _ = w.shape
    offsets, order = plan(bqm, ids, groups)
    y = torch.full((len(ids), n // 2 if glu else n), 77.0, dtype=TYPES[t], device=DEV)
    return bqm.bqm_mxfp4_grouped_gemm(dev(w), dev(ws), dev(xq), dev(xs), offsets, order, glu=glu, y=y)


def check_gemm(bqm, w, ws, xq, xs, ids, glu, t="f32"):
    k = 2 * w.shape[2]
    y = gemm(bqm, w, ws, xq, xs, ids, glu, t).cpu().double().numpy()
    p, total = groups_ref.expert_products(w, ws, layer_ref.mxfp4_values(xq, xs), ids, len(ids) // len(xq))
    want, tol = p, (3 * k / 64 + 2) * 2.0 ** -23 * total
    if glu:
        want, tol = groups_ref.gated(p, tol)
    # fp16: from 65520 on (its largest value and half a step) the nearest is infinite
    past = np.isinf(y) & (np.sign(y) == np.sign(want)) & (np.abs(want) + tol >= 65520) if t == "f16" else False
    tol = with_type(want, tol, t)
    none = (ids < 0) | (ids >= w.shape[0])
    assert (y[none] == 0).all()
    y = np.where(past, want, y)
    assert (np.abs(y - want)[~none] <= tol[~none]).all(), (np.abs(y - want)[~none] / tol[~none]).max()


SHAPES = [  # rows, top, groups, k, n
    (1, 1, 1, 32, 2), (1, 2, 4, 64, 34), (3, 2, 5, 96, 66), (16, 4, 8, 288, 130), (40, 2, 3, 1024, 64),
    (65, 3, 4, 1056, 258), (7, 8, 64, 2048, 96), (200, 1, 3, 512, 514), (333, 2, 2, 1440, 320), (130, 6, 100, 544, 190),
    (20, 1, 1024, 256, 36), (500, 4, 1, 128, 70), (64, 8, 16, 4128, 128), (300, 4, 16, 800, 1030),
    # few tiles and long rows: the kernel whose waves share k
    (16, 2, 8, 4096, 130), (5, 3, 4, 8224, 66), (33, 1, 2, 16416, 50), (100, 1, 2, 2080, 200), (1, 3, 4, 4064, 34),
    # more tiles of 128 x 128 than a card takes at once: the large tile
    (300, 2, 64, 544, 2080), (1500, 1, 5, 800, 5150), (700, 2, 3, 288, 6002), (90, 1, 90, 1056, 1602),
]


@pytest.mark.parametrize("rows,top,groups,k,n", SHAPES)
@pytest.mark.parametrize("glu,t", [(False, "f32"), (True, "f32"), (True, "bf16"), (False, "f16")])
def test_grouped_gemm(bqm, rows, top, groups, k, n, glu, t):
    rng = np.random.default_rng(rows * 7 + k)
    low, high = (122, 126) if glu else (118, 132)
    w, ws = random_mx((groups, n), k, rng, low, high)
    xq, xs = random_mx((rows,), k, rng, low, high)
    ids = rng.integers(-1, groups + 1, rows * top)
    check_gemm(bqm, w, ws, xq, xs, ids, glu, t)


@pytest.mark.parametrize("kind", ["one", "last", "none", "two", "steps"])
@pytest.mark.parametrize("glu", [False, True])
def test_grouped_gemm_distributions(bqm, kind, glu):
    """Everything to one expert, to none, or as many rows to each as fill tiles exactly, or all but one."""
    rng = np.random.default_rng(5)
    groups, k, n, slots = 6, 320, 132, 520
    ids = {"one": np.zeros(slots, int), "last": np.full(slots, groups - 1), "none": np.full(slots, -1),
           "two": np.where(rng.random(slots) < 0.5, 1, 4),
           "steps": np.repeat([0, 1, 2, 3, 4, 5, -1], [16, 64, 65, 128, 127, 1, slots - 401])}[kind]
    w, ws = random_mx((groups, n), k, rng, 122, 126)
    xq, xs = random_mx((slots // 2 if kind != "steps" else slots,), k, rng, 122, 126)
    check_gemm(bqm, w, ws, xq, xs, rng.permutation(ids), glu)


@pytest.mark.parametrize("n", [1, 33, 255, 4098])
@pytest.mark.parametrize("glu", [False, True])
def test_grouped_gemm_every_count_of_rows(bqm, n, glu):
    """Groups of 1, 31, 32, 33 .. 300 rows, of every type, in the small tile and (the widest n) in the large one."""
    if glu:
        n *= 2
    rng = np.random.default_rng(n)
    counts = [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 300, 0, 2]
    ids = rng.permutation(np.repeat(np.arange(len(counts)), counts))
    k = 96
    w, ws = random_mx((len(counts), n), k, rng, 122, 126)
    xq, xs = random_mx((len(ids),), k, rng, 122, 126)
    for t in TYPES:
        check_gemm(bqm, w, ws, xq, xs, ids, glu, t)


@pytest.mark.parametrize("rows,top,groups,n,k", [(24, 4, 8, 200, 1056), (24, 4, 8, 200, 5152), (400, 2, 4, 200, 1056),
                                                 (1500, 2, 3, 200, 1056), (1500, 2, 3, 2600, 1056)])
def test_grouped_gemm_a_slots_bits_do_not_depend_on_the_others(bqm, rows, top, groups, n, k):
    rng = np.random.default_rng(8)
    w, ws = random_mx((groups, n), k, rng, 100, 150)
    xq, xs = random_mx((rows,), k, rng, 100, 150)
    ids = rng.integers(0, groups, rows * top)
    other = rng.integers(0, groups, rows * top)
    kept = rng.permutation(rows * top)[: rows * top // 2]
    other[kept] = ids[kept]
    a, b = gemm(bqm, w, ws, xq, xs, ids, False), gemm(bqm, w, ws, xq, xs, other, False)
    assert torch.equal(a[kept].view(torch.int32), b[kept].view(torch.int32))


@pytest.mark.parametrize("k", [32, 96, 800, 1024, 1056, 1440, 4128, 8192])
def test_grouped_gemm_nan_scales_stay_with_their_rows(bqm, k):
    """A scale byte 255 makes its slot or weight row NaN, and nothing beside it: not the rows whose scales follow."""
    rng = np.random.default_rng(k)
    groups, n, rows = 3, 70, 150
    w, ws = random_mx((groups, n), k, rng)
    xq, xs = random_mx((rows,), k, rng)
    ids = rng.integers(0, groups, rows)
    ws[1, 5, :], ws[2, n - 1, -1], xs[7, 0], xs[33, -1] = 255, 255, 255, 255
    y = gemm(bqm, w, ws, xq, xs, ids, False).isnan().cpu().numpy()
    want = np.zeros_like(y)
    want[ids == 1, 5], want[ids == 2, n - 1], want[7], want[33] = True, True, True, True
    assert np.array_equal(y, want)


@pytest.mark.parametrize("rows,n,k", [(40, 70, 1056), (40, 70, 4128), (300, 6200, 544)])
def test_grouped_gemm_every_scale_byte(bqm, rows, n, k):
    """Scale bytes over their whole range, those of a block's two sides near a sum of 254, so that results are near 1;
    k ends inside a stage, and what stands there must not count."""
    rng = np.random.default_rng(k)
    groups = 3
    w, xq = (rng.integers(0, 256, shape).astype(np.uint8) for shape in ((groups, n, k // 2), (rows, k // 2)))
    at = rng.permutation(np.arange(k // 32) * 254 // (k // 32 - 1))
    xs = np.clip(at[None, :] + rng.integers(-2, 3, (rows, k // 32)), 0, 254).astype(np.uint8)
    ws = np.clip(254 - at[None, None, :] + rng.integers(-2, 3, (groups, n, k // 32)), 0, 254).astype(np.uint8)
    check_gemm(bqm, w, ws, xq, xs, rng.integers(0, groups, rows), False)


@pytest.mark.parametrize("k", [1056, 8160])
def test_expert_gemv_every_scale_byte(bqm, k):
    rng = np.random.default_rng(k)
    w = rng.integers(0, 256, (2, 50, k // 2)).astype(np.uint8)
    at = rng.permutation(np.arange(k // 32) * 252 // (k // 32 - 1))
    ws = np.clip(at[None, None, :] + rng.integers(-2, 3, (2, 50, k // 32)), 0, 252).astype(np.uint8)
    # x of a block brings its terms near 1, as far as its own bits reach
    x = rng.standard_normal((6, k)) * np.exp2(np.clip(127.0 - np.repeat(at, 32), -100, 120))
    check_gemv(bqm, w, ws, x.astype(np.float32), np.array([0, 1, 0, 0, 1, 1]), False)


def test_grouped_gemm_bad_entries_are_passed_over(bqm):
    """Order entries and offsets outside the slots lead nowhere: the good rows come out right, nothing else is touched."""
    rng = np.random.default_rng(4)
    groups, k, n, slots = 4, 256, 40, 60
    w, ws = random_mx((groups, n), k, rng)
    xq, xs = random_mx((slots,), k, rng)
    ids = rng.integers(0, groups, slots)
    offsets, order = plan(bqm, ids, groups)
    good = bqm.bqm_mxfp4_grouped_gemm(dev(w), dev(ws), dev(xq), dev(xs), offsets, order)
    bad = order.clone()
    lost = order[[3, 20, 41]].long()
    bad[3], bad[20], bad[41] = -1, slots, 2 ** 31 - 1
    y = torch.full((slots, n), 77.0, device=DEV)
    bqm.bqm_mxfp4_grouped_gemm(dev(w), dev(ws), dev(xq), dev(xs), offsets, bad, y=y)
    keep = torch.ones(slots, dtype=torch.bool, device=DEV)
    keep[lost] = False
    assert torch.equal(y[keep], good[keep]) and bool((y[lost] == 77).all())
    ends = offsets.clone()
    ends[-1] = 2 ** 31 - 1
    ends[0] = -5
    assert torch.equal(bqm.bqm_mxfp4_grouped_gemm(dev(w), dev(ws), dev(xq), dev(xs), ends, order), good)


def test_grouped_gemm_offsets_that_are_none_touch_nothing_else(bqm):
    """Groups that overlap, run backwards or all hold everything: whatever the outputs are, they stay in their tensor."""
    rng = np.random.default_rng(9)
    groups, k, n, slots = 300, 64, 34, 700
    w, ws = random_mx((groups, n), k, rng)
    xq, xs = random_mx((slots,), k, rng)
    order = dev(rng.permutation(slots).astype(np.int32))
    for kind in ("all", "backwards", "wild"):
        offsets = {"all": np.arange(groups + 1) % 2 * slots, "backwards": np.linspace(slots, 0, groups + 1),
                   "wild": rng.integers(-2 ** 31, 2 ** 31, groups + 1)}[kind].astype(np.int32)
        wide = torch.full((slots + 2, n), 77.0, device=DEV)
        bqm.bqm_mxfp4_grouped_gemm(dev(w), dev(ws), dev(xq), dev(xs), dev(offsets), order, y=wide[1:-1])
        assert bool((wide[0] == 77).all()) and bool((wide[-1] == 77).all()) and bool(wide[1:-1].isfinite().all())


def check_gemv(bqm, w, ws, x, ids, glu):
    k, slots = x.shape[1], len(ids)
    n = w.shape[1]
    y = torch.full((slots, n // 2 if glu else n), 77.0, device=DEV)
    bqm.bqm_mxfp4_expert_gemv(dev(w), dev(ws), dev(x), dev(ids.astype(np.int32)), glu, y)
    p, total = groups_ref.expert_products(w, ws, x.astype(np.float64), ids, slots // len(x))
    want, tol = p, (8 * 16 * -(-(-(-k // 512)) // 8) + 8 + 4) * 2.0 ** -23 * total
    if glu:
        want, tol = groups_ref.gated(p, tol)
    got = y.cpu().double().numpy()
    none = (ids < 0) | (ids >= w.shape[0])
    assert (got[none] == 0).all()
    assert (np.abs(got - want)[~none] <= tol[~none]).all(), (np.abs(got - want)[~none] / tol[~none]).max()
    return y


@pytest.mark.parametrize("rows,top,groups,k,n", [
    (1, 1, 1, 32, 2), (1, 4, 8, 256, 66), (1, 8, 32, 4096, 130), (2, 2, 4, 96, 34), (3, 6, 4, 1408, 96),
    (5, 1, 1, 1024, 64), (6, 1, 1, 544, 40), (16, 8, 16, 512, 72), (16, 16, 20, 160, 50), (9, 6, 64, 1440, 100),
    (11, 2, 2, 4128, 38), (4, 3, 3, 8224, 36), (2, 2, 2, 16384, 34), (256, 1, 1000, 64, 10), (1, 2, 1024, 2880, 514)])
@pytest.mark.parametrize("glu", [False, True])
def test_expert_gemv(bqm, rows, top, groups, k, n, glu):
    rng = np.random.default_rng(rows + k)
    w, ws = random_mx((groups, n), k, rng, 118, 124)
    x = rng.standard_normal((rows, k)).astype(np.float32)
    ids = rng.integers(-1, groups + 1, rows * top)
    check_gemv(bqm, w, ws, x, ids, glu)


@pytest.mark.parametrize("k", [320, 4096])
def test_expert_gemv_bits_do_not_depend_on_the_other_slots(bqm, k):
    """Alone, among others of its expert at any place, and among other experts: the same bits."""
    rng = np.random.default_rng(k)
    groups, n = 5, 70
    w, ws = random_mx((groups, n), k, rng, 90, 160)
    x = (rng.standard_normal((12, k)) * np.exp2(rng.integers(-20, 20, (12, k)))).astype(np.float32)
    runs = [np.zeros(12, int), np.array([0, 1, 0, 2, 0, 3, 0, 4, 0, 1, 0, 0]), rng.integers(0, 2, 12)]
    ys = [bqm.bqm_mxfp4_expert_gemv(dev(w), dev(ws), dev(x), dev(r.astype(np.int32))) for r in runs]
    for r, y in zip(runs[1:], ys[1:]):
        at = np.nonzero(r == 0)[0]
        assert torch.equal(y[at].view(torch.int32), ys[0][at].view(torch.int32))


def test_expert_gemv_infinity_and_nan_stay_with_their_slot(bqm):
    rng = np.random.default_rng(3)
    w, ws = random_mx((2, 40), 256, rng)
    x = rng.standard_normal((7, 256)).astype(np.float32)
    x[2, 5], x[4, 200], x[6, 0] = np.inf, np.nan, -np.inf
    y = bqm.bqm_mxfp4_expert_gemv(dev(w), dev(ws), dev(x), dev(np.zeros(7, np.int32))).cpu()
    assert not bool(y[[2, 4, 6]].isfinite().all(1).any()) and bool(y[[0, 1, 3, 5]].isfinite().all())


def test_expert_gemv_is_the_gemv_of_its_expert(bqm):
    """One slot against the product with that expert's matrix alone, within both tolerances."""
    rng = np.random.default_rng(6)
    w, ws = random_mx((3, 96), 2048, rng, 118, 124)
    x = rng.standard_normal((1, 2048)).astype(np.float32)
    y = check_gemv(bqm, w, ws, x, np.array([2]), False)
    one = bqm.bqm_mxfp4_gemv(dev(w[2]), dev(ws[2]), dev(x))
    _, total = layer_ref.mxfp4_matmul(w[2], ws[2], x.astype(np.float64))
    assert (np.abs((y - one).cpu().numpy()) <= 2 * 140 * 2.0 ** -23 * total).all()


def test_experts_past_4_gib(bqm):
    """Weights of more than 4 GiB: the last expert's, against the same matrix alone."""
    groups, n, k = 600, 4096, 4096
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.randint(0, 256, (groups, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    ws = torch.randint(118, 122, (groups, n, k // 32), generator=g, device=DEV, dtype=torch.uint8)
    xq = torch.randint(0, 256, (20, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    xs = torch.randint(124, 128, (20, k // 32), generator=g, device=DEV, dtype=torch.uint8)
    ids = torch.tensor([0, 255, 256, 511, 512, 599, 599, 300, 599, 7], dtype=torch.int32, device=DEV).repeat(2)
    offsets, order = bqm.bqm_group_rows(ids, groups)
    y = bqm.bqm_mxfp4_grouped_gemm(w, ws, xq, xs, offsets, order)
    x = bqm.bqm_mxfp4_dequantize(xq, xs)
    z = bqm.bqm_mxfp4_expert_gemv(w, ws, x, ids)
    for e in ids.unique().tolist():
        at = (ids == e).nonzero()[:, 0]
        v = bqm.bqm_mxfp4_dequantize(w[e], ws[e]).double()
        want, total = x[at].double() @ v.t().contiguous(), x[at].double().abs() @ v.abs().t().contiguous()
        assert bool(((y[at] - want).abs() <= (3 * k / 64 + 2) * 2.0 ** -23 * total).all())
        assert bool(((z[at] - want).abs() <= 140 * 2.0 ** -23 * total).all())


def test_outputs_past_4_gib(bqm):
    """More than 2^31 outputs and 2^31 bytes of x: rows either side of the marks, and the last."""
    slots, k, n = 1_100_003, 32, 2048
    g = torch.Generator(device=DEV).manual_seed(2)
    w = torch.randint(0, 256, (3, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    ws = torch.randint(118, 132, (3, n, 1), generator=g, device=DEV, dtype=torch.uint8)
    xq = torch.randint(0, 256, (slots, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    xs = torch.randint(118, 132, (slots, 1), generator=g, device=DEV, dtype=torch.uint8)
    ids = torch.randint(0, 3, (slots,), generator=g, device=DEV, dtype=torch.int32)
    offsets, order = bqm.bqm_group_rows(ids, 3)
    y = bqm.bqm_mxfp4_grouped_gemm(w, ws, xq, xs, offsets, order)
    marks = [0, 1, 2 ** 19 - 1, 2 ** 19, 2 ** 19 + 1, 2 ** 20 - 1, 2 ** 20, 2 ** 20 + 1, slots - 2, slots - 1]
    x = bqm.bqm_mxfp4_dequantize(xq[marks], xs[marks]).double()
    for i, s in enumerate(marks):
        v = bqm.bqm_mxfp4_dequantize(w[ids[s]], ws[ids[s]]).double()
        want, total = v @ x[i], v.abs() @ x[i].abs()
        assert bool(((y[s] - want).abs() <= 4 * 2.0 ** -23 * total).all()), s
