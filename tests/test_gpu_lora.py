"""Low-rank adapters against 64 bits.

Tolerance, H = sum |x| |A|, T = sum_r H |B|, on every output.  x or h of f32 has three parts and an fp16 adapter two;
their magnitudes sum to at most 1.02 of the value's.  A 32-k step of P products of parts adds at most 8 P times, cut, 2^-23
each; a wave has one in eight of k's steps, then come the waves; h's f32 has one step a 32 ranks:
  |h - exact| <= th H,  th = 1.02 (8 P ceil(k / 256) + 8) 2^-23;
  |y - exact| <= |scale| T (th + 1.02 * 8 P' ceil(r / 32) 2^-23 + 2^-24) + 2^-24 |y|.
"""
import numpy as np
import pytest


pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
PAIRS = [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")]
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_02_amd as m

    m.lib()
    return m


def make(m, k, n, r, adapters, xt, abt, seed=0, spread=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k), generator=g)
    if spread:
        x = torch.ldexp(x, torch.randint(-spread, spread, (m, k), generator=g))
    a = torch.randn((adapters, r, k), generator=g) / k ** 0.5
    b = torch.randn((adapters, n, r), generator=g) * 0.2
    return x.to(TYPES[xt]).to(DEV), a.to(TYPES[abt]).to(DEV), b.to(TYPES[abt]).to(DEV)


def reference(x, a, b, ids, scale, res, xt, abt):
    x, a, b = (v.cpu().double().numpy() for v in (x, a, b))
    m, k, n, r = len(x), x.shape[1], b.shape[1], a.shape[1]
    y, tol = np.zeros((m, n)), np.zeros((m, n))
    p1 = (3 if xt == "f32" else 1) * (2 if abt == "f16" and xt == "f32" else 1)
    p2 = 3 * (2 if abt == "f16" else 1)
    th = 1.02 * (8 * p1 * -(-k // 256) + 8) * 2.0 ** -23
    te = 1.02 * 8 * p2 * -(-r // 32) * 2.0 ** -23
    for e in range(len(a)):
        at = np.nonzero(ids == e)[0]
        s = 1.0 if scale is None else float(scale[e])
        y[at] = s * ((x[at] @ a[e].T) @ b[e].T)
        tol[at] = abs(s) * (np.abs(x[at]) @ np.abs(a[e]).T) @ np.abs(b[e]).T * (th + te + 2.0 ** -24)
    if res is not None:
        y = y + res.cpu().double().numpy()
    return y, tol + 2.0 ** -24 * np.abs(y)


def check(bqm, x, a, b, ids, scale, res, xt, abt, in_place=False, ldy=0):
    m, n, adapters = len(x), b.shape[1], len(a)
    offsets, order = bqm.bqm_group_rows(torch.from_numpy(ids.astype(np.int32)).to(DEV), adapters)
    want, tol = reference(x, a, b, ids, scale, res, xt, abt)
    wide = torch.full((m, max(ldy, n)), 77.0, device=DEV)
    if in_place:
        wide[:, :n] = res
    y = wide[:, :n]
    need = bqm.bqm_lora_add_workspace(m, a.shape[1])
    work = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    bqm.bqm_lora_add(x, a, b, offsets, order, scale, y if in_place else res, y, work)
    got = wide.cpu().double().numpy()
    err = np.abs(got[:, :n] - want)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()
    assert (got[:, n:] == 77).all() and bool((work[need:] == 0x5A).all())
    none = (ids < 0) | (ids >= adapters)
    assert np.array_equal(got[none, :n], np.zeros((none.sum(), n)) if res is None else res.cpu().double().numpy()[none])
    return y


@pytest.mark.parametrize("xt,abt", PAIRS)
@pytest.mark.parametrize("m,k,n,r,adapters", [
    (1, 8, 1, 8, 1), (1, 256, 4, 16, 3), (3, 264, 66, 8, 2), (17, 1024, 255, 16, 4), (40, 520, 257, 24, 1),
    (64, 4096, 130, 16, 64), (33, 96, 1030, 40, 5), (100, 1000, 300, 64, 3), (50, 2048, 90, 128, 7), (20, 136, 70, 256, 2),
    (300, 264, 515, 72, 4), (15, 40, 33, 160, 1024), (600, 512, 200, 32, 2)])
def test_lora_add(bqm, xt, abt, m, k, n, r, adapters):
    rng = np.random.default_rng(m + k)
    x, a, b = make(m, k, n, r, adapters, xt, abt, seed=k)
    scale = torch.from_numpy((0.5 + rng.random(adapters)).astype(np.float32)).to(DEV)
    res = torch.randn((m, n), generator=torch.Generator().manual_seed(1)).to(DEV)
    ids = rng.integers(-1, adapters + 1, m)
    check(bqm, x, a, b, ids, scale, res, xt, abt)
    check(bqm, x, a, b, ids, None, None, xt, abt, ldy=n + 3)


@pytest.mark.parametrize("n,ldy", [(64, 0), (64, 100), (64, 65), (37, 41)])
def test_lora_add_in_place_in_a_wider_buffer(bqm, n, ldy):
    rng = np.random.default_rng(n)
    x, a, b = make(50, 128, n, 16, 3, "f32", "bf16")
    res = torch.randn((50, n), generator=torch.Generator().manual_seed(1)).to(DEV)
    check(bqm, x, a, b, rng.integers(-1, 3, 50), None, res, "f32", "bf16", in_place=True, ldy=ldy)


def test_lora_add_strided_x_and_res(bqm):
    rng = np.random.default_rng(2)
    for xt, abt in PAIRS:
        x, a, b = make(21, 192 + 64, 50, 16, 2, xt, abt)
        a = a[:, :, :192].contiguous()
        res = torch.randn((42, 61), generator=torch.Generator().manual_seed(1)).to(DEV)[::2, 5:55]
        check(bqm, x[:, 32:224], a, b, rng.integers(-1, 2, 21), None, res, xt, abt)


@pytest.mark.parametrize("kind", ["one", "none", "runs", "each"])
def test_lora_add_distributions(bqm, kind):
    rng = np.random.default_rng(7)
    m, adapters = 130, 130
    ids = {"one": np.full(m, 5), "none": np.full(m, -1), "runs": np.repeat([3, -1, 129, 0], [64, 1, 16, 49]), "each": rng.permutation(m)}[kind]
    x, a, b = make(m, 256, 100, 16, adapters, "f32", "bf16")
    res = torch.randn((m, 100), generator=torch.Generator().manual_seed(1)).to(DEV)
    check(bqm, x, a, b, ids, None, res, "f32", "bf16")


@pytest.mark.parametrize("abt", ["bf16", "f16"])
def test_lora_add_f32_operands_are_not_rounded(bqm, abt):
    """x over 40 binades: the bound of f32 sums holds, which parts lost or rounded would break."""
    x, a, b = make(30, 512, 64, 16, 2, "f32", abt, spread=20)
    check(bqm, x, a, b, np.arange(30) % 2, None, None, "f32", abt)
    # one term: h is the product, y the product of that, each rounded once (16 significant bits fit an f32)
    x = torch.zeros((4, 64), device=DEV)
    x[:, 9] = torch.tensor([1 + 2.0 ** -23, 3.1415927, 1e-20, 1e20], device=DEV)
    a = torch.zeros((1, 8, 64), dtype=TYPES[abt], device=DEV)
    b = torch.zeros((1, 5, 8), dtype=TYPES[abt], device=DEV)
    a[0, 3, 9], b[0, 2, 3] = 1.0, 1.0
    off, order = bqm.bqm_group_rows(torch.zeros(4, dtype=torch.int32, device=DEV), 1)
    y = bqm.bqm_lora_add(x, a, b, off, order)
    assert torch.equal(y[:, 2], x[:, 9]) and float(y.abs().sum()) == float(x.abs().sum())


def test_lora_add_bits_do_not_depend_on_the_other_rows(bqm):
    x, a, b = make(60, 520, 70, 24, 3, "f32", "bf16", spread=8)
    rng = np.random.default_rng(5)
    ids, other = rng.integers(0, 3, 60), rng.integers(0, 3, 60)
    other[::2] = ids[::2]

    def run(i):
        off, order = bqm.bqm_group_rows(torch.from_numpy(i.astype(np.int32)).to(DEV), 3)
        return bqm.bqm_lora_add(x, a, b, off, order)

    assert torch.equal(run(ids)[::2].view(torch.int32), run(other)[::2].view(torch.int32))


def test_lora_add_infinity_and_nan_stay_with_their_row(bqm):
    for xt, abt in PAIRS:
        x, a, b = make(20, 128, 40, 8, 1, xt, abt)
        x[3, 7], x[11, 100] = float("inf"), float("nan")
        off, order = bqm.bqm_group_rows(torch.zeros(20, dtype=torch.int32, device=DEV), 1)
        y = bqm.bqm_lora_add(x, a, b, off, order).isfinite()
        rows = torch.ones(20, dtype=torch.bool, device=DEV)
        rows[[3, 11]] = False
        assert bool(y[rows].all()) and not bool(y[[3, 11]].any())


def test_lora_add_nan_in_another_adapter_or_past_the_rank(bqm):
    x, a, b = make(20, 136, 40, 8, 3, "f32", "bf16")
    a[1], b[1] = float("nan"), float("nan")
    ids = np.array([0, 2] * 10)
    check(bqm, x, torch.nan_to_num(a), torch.nan_to_num(b), ids, None, None, "f32", "bf16")
    off, order = bqm.bqm_group_rows(torch.from_numpy(ids.astype(np.int32)).to(DEV), 3)
    clean = bqm.bqm_lora_add(x, torch.nan_to_num(a), torch.nan_to_num(b), off, order)
    assert torch.equal(bqm.bqm_lora_add(x, a, b, off, order), clean)


def test_lora_add_bad_entries_are_passed_over(bqm):
    x, a, b = make(40, 64, 30, 8, 2, "f32", "bf16")
    off, order = bqm.bqm_group_rows((torch.arange(40, device=DEV) % 3).int(), 2)
    good = bqm.bqm_lora_add(x, a, b, off, order)
    bad, lost = order.clone(), order[[2, 17, 39]].long()
    bad[2], bad[17], bad[39] = -1, 40, 2 ** 31 - 1
    y = torch.full((40, 30), 77.0, device=DEV)
    bqm.bqm_lora_add(x, a, b, off, bad, y=y)
    keep = torch.ones(40, dtype=torch.bool, device=DEV)
    keep[lost] = False
    assert torch.equal(y[keep], good[keep]) and bool((y[lost] == 77).all())


@pytest.mark.parametrize("m,adapters,r", [(1024, 16, 16), (1100, 3, 24), (3300, 4, 64), (1030, 2, 136), (6200, 2, 8), (12400, 1, 72)])
def test_lora_add_many_rows(bqm, m, adapters, r):
    """Adapters of many rows: 64 rows a workgroup, k in eight, four, two and one part."""
    rng = np.random.default_rng(m)
    for xt, abt in PAIRS:
        x, a, b = make(m, 264, 70, r, adapters, xt, abt, seed=m)
        ids = rng.integers(-1, adapters, m)
        res = torch.randn((m, 70), generator=torch.Generator().manual_seed(1)).to(DEV)
        check(bqm, x, a, b, ids, None, res, xt, abt)


def test_lora_add_past_4_gib(bqm):
    """y of more than 2^31 values in a wide buffer: rows either side of the marks."""
    m, n, ldy = 70_000, 64, 33_000
    x, a, b = make(m, 64, n, 8, 3, "bf16", "bf16")
    wide = torch.zeros((m, ldy), device=DEV)
    ids = (np.arange(m) % 4) - 1
    off, order = bqm.bqm_group_rows(torch.from_numpy(ids.astype(np.int32)).to(DEV), 3)
    y = wide[:, 7:7 + n]
    bqm.bqm_lora_add(x, a, b, off, order, res=y, y=y)
    want, tol = reference(x, a, b, ids, None, None, "bf16", "bf16")
    assert (np.abs(y.cpu().double().numpy() - want) <= tol).all()
    assert float(wide[:, :7].abs().max()) == 0 and float(wide[:, 7 + n:].abs().max()) == 0
