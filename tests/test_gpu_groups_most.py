"""The operators of include/bqmm_groups.h at the largest sizes that they take, on rows either side of the marks where a
32-bit count or offset would wrap, against 64 bits (tolerances as in test_gpu_grouped)."""
import numpy as np
import pytest

import layer_ref
import test_gpu_lora as lora

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_02_amd as m

    m.lib()
    yield m
    torch.cuda.empty_cache()


@pytest.mark.parametrize("glu,n", [(False, 2 ** 31 - 1025), (False, 2 ** 31 - 513), (False, 2 ** 31 - 32), (False, 2 ** 31 - 1), (True, 2 ** 31 - 2)])
def test_expert_gemv_the_most_weight_rows(bqm, glu, n):
    """34 GB of codes; a second slot of no expert, all zeros to the last output.  Rounded up to units of 32 rows the
    largest n leave 31 bits, and the last 512 outputs end a workgroup's steps past them."""
    k, outs = 32, n // 2 if glu else n
    w = torch.full((1, n, k // 2), 0x22, dtype=torch.uint8, device=DEV)
    ws = torch.full((1, n, 1), 122, dtype=torch.uint8, device=DEV)
    at = torch.tensor([0, 1, 2 ** 26 - 1, 2 ** 26, 2 ** 27, 2 ** 28 - 1, 2 ** 28, 2 ** 29 - 1, 2 ** 29, 2 ** 30 - 33,
                       outs - 1056, outs - 1025, outs - 1024, outs - 513, outs - 34, outs - 33, outs - 32, outs - 17,
                       outs - 16, outs - 2, outs - 1] + ([] if glu else [2 ** 30 - 1, 2 ** 30, 2 ** 30 + 1, 2 ** 31 - 2048])).unique()
    rng = np.random.default_rng(5)
    rows = torch.cat((at, at + outs)) if glu else at
    codes = rng.integers(0, 256, (len(rows), k // 2)).astype(np.uint8)
    w[0, rows.to(DEV)] = torch.from_numpy(codes).to(DEV)
    x = rng.standard_normal((2, k)).astype(np.float32)
    y = torch.full((2, outs), 77.0, device=DEV)
    bqm.bqm_mxfp4_expert_gemv(w, ws, torch.from_numpy(x).to(DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV), glu, y)
    v = layer_ref.mxfp4_values(codes, np.full((len(rows), 1), 122, np.uint8))
    p, total = v @ x[0].astype(np.float64), np.abs(v) @ np.abs(x[0].astype(np.float64))
    tol = (8 * 16 + 8 + 4) * 2.0 ** -23 * total
    if glu:
        import groups_ref

        p, tol = (r[0] for r in groups_ref.gated(p[None], tol[None]))
    got = y[0, at.to(DEV)].cpu().double().numpy()
    assert (np.abs(got - p) <= tol).all()
    assert int(torch.count_nonzero(y[1])) == 0
    # every other row has the same weights: 32 ones of 2^-5
    ones = float(x[0].astype(np.float64).sum() / 32)
    want = ones / (1 + np.exp(-ones)) * ones if glu else ones
    rest = y[0]
    rest[at.to(DEV)] = float(rest[3])
    assert float(rest.max()) == float(rest.min()) and abs(float(rest[3]) - want) <= 200 * 2.0 ** -23 * np.abs(x[0]).sum() / 32 * (1 + abs(ones))


@pytest.mark.parametrize("m,adapters,k,n,r,xt,abt", [(600_001, 40, 64, 70, 24, "bf16", "bf16"), (2_097_087, 1, 16, 5, 8, "f32", "f16")])
def test_lora_add_the_most_rows(bqm, m, adapters, k, n, r, xt, abt):
    """More than the half million rows that any rank and width once had to keep below, and as many as a grid has."""
    rng = np.random.default_rng(m)
    x, a, b = lora.make(m, k, n, r, adapters, xt, abt)
    res = torch.randn((m, n), generator=torch.Generator().manual_seed(1)).to(DEV)
    lora.check(bqm, x, a, b, rng.integers(-1, adapters, m), None, res, xt, abt)


# tiles of 256 rows; of 128 (the most bytes of x); of 256 at that; the waves that share k
@pytest.mark.parametrize("rows,k,n", [(900_001, 8192, 64), (8191, 2 ** 20, 32), (8191, 2 ** 20, 1100), (5000, 2 ** 20, 32)])
def test_grouped_gemm_x_past_2_gib(bqm, rows, k, n):
    """x of 2.6 to 4.3 GB.  A row of x has one block that is not zeros, so its sums are exact: rows either side of 2 GiB,
    the last ones and others."""
    nblk = k // 32
    g = torch.Generator(device=DEV).manual_seed(rows)
    w = torch.randint(0, 256, (1, n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    ws = torch.randint(120, 134, (1, n, nblk), generator=g, device=DEV, dtype=torch.uint8)
    xq = torch.zeros((rows, nblk, 16), dtype=torch.uint8, device=DEV)
    xs = torch.full((rows, nblk), 127, dtype=torch.uint8, device=DEV)
    block = torch.arange(rows, device=DEV) * 7919 % nblk
    codes = torch.randint(0, 256, (rows, 16), generator=g, device=DEV, dtype=torch.uint8)
    xq[torch.arange(rows, device=DEV), block] = codes
    offsets = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    order = torch.randperm(rows, generator=g, device=DEV).int()
    y = bqm.bqm_mxfp4_grouped_gemm(w, ws, xq.view(rows, k // 2), xs, offsets, order)
    mark = 2 ** 31 // (k // 2)
    at = sorted({0, 1, mark - 1, mark, mark + 1, rows - 2, rows - 1, *np.random.default_rng(k).integers(0, rows, 120).tolist()})
    for r in at:
        b = int(block[r])
        v = layer_ref.mxfp4_values(w[0, :, 16 * b:16 * b + 16].cpu().numpy(), ws[0, :, b:b + 1].cpu().numpy())
        x = layer_ref.mxfp4_values(codes[r:r + 1].cpu().numpy(), np.full((1, 1), 127, np.uint8))[0]
        assert np.array_equal(y[r].cpu().double().numpy(), v @ x), r
