"""The norms with 8-bit outputs on rows of infinities, NaN, zeros and values at the ends of f32: what the norm and the
quantizer give in two calls, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_02_amd as m

    m.lib()
    return m


def rows(k, t):
    g = torch.Generator().manual_seed(k)
    x = torch.randn((12, k), generator=g)
    x[0] = 0
    x[1, k // 2] = float("inf")
    x[2, 7] = float("nan")
    x[3] = float("nan")
    x[4] = 0
    x[4, k - 1] = 3.0                  # one value in a row of zeros
    x[5] *= 1e-30
    x[6, ::2] = 0
    x[7, 3] = 3e4                      # one outlier
    x[8] = -x[8].abs()
    x[9] = 1.0
    x[10, 0], x[10, 1] = float("inf"), -float("inf")
    x[11, -32:] = 0
    return x.to(t).to(DEV)


def same(a, b):
    a, b = a.view(torch.int32), b.view(torch.int32)
    nan = (a & 0x7FFFFFFF) > 0x7F800000
    return torch.equal(nan, (b & 0x7FFFFFFF) > 0x7F800000) and torch.equal(a[~nan], b[~nan])


@pytest.mark.parametrize("t", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("k", [32, 160, 4096, 5152, 20480])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_special_rows_are_what_two_calls_give(bqm, k, t, eps):
    x = rows(k, t)
    g = torch.Generator().manual_seed(1)
    gain = 1.0 + 0.1 * torch.randn(k, generator=g)
    gain[1], gain[2], gain[k - 1] = 1e38, 1e-38, 0.0       # y at the ends of f32
    gain = gain.to(DEV)
    for gn in (None, gain):
        y, _ = bqm.bqm_add_rmsnorm(x, None, gn, eps)
        q, d = bqm.bqm_q8_1_quantize(y)
        nq, nd, _ = bqm.bqm_add_rmsnorm_q8_1(x, None, gn, eps)
        assert torch.equal(nq, q) and same(nd, d)
        e, s = bqm.bqm_e4m3_blk_quantize(y)
        ne, ns, _ = bqm.bqm_add_rmsnorm_e4m3_blk(x, None, gn, eps)
        assert torch.equal(ne, e) and same(ns, s)
