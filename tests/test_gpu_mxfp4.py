"""MXFP4: quantization and dequantization bit for bit, the two products against 64 bits.

Tolerances, T = sum |terms|, on every output:
* GEMM: the products of a 32-block share one power of two and are multiples of
  a quarter up to 36, so a block's sum is exact; each 64-k step adds two block
  sums to the accumulator, at most three cut or rounded additions of 2^-23:
  (3 k / 64 + 2) 2^-23 T.
* GEMV: exact products (bf16 x bf16), three operand rows per token; a 32-k
  step sums 32 products and the accumulator, at most eight cut additions; 16
  steps per wave, then the waves, passes and three parts:
  (8 * 16 + ceil(k / 512) + 4) 2^-23 T.
"""
import numpy as np
import pytest

import layer_ref

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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def random_mx(rows, k, rng, low=118, high=132):
    return (rng.integers(0, 256, (rows, k // 2)).astype(np.uint8),
            rng.integers(low, high, (rows, k // 32)).astype(np.uint8))


def same_bits(a, b):
    return np.array_equal(a.view(np.uint32), b.view(np.uint32))


def quantize(bqm, x):
    m, k = x.shape
    codes = torch.full((m, k // 2), 0x99, dtype=torch.uint8, device=DEV)
    scales = torch.full((m, k // 32), 0x99, dtype=torch.uint8, device=DEV)
    bqm.bqm_mxfp4_quantize(x, codes, scales)
    return codes.cpu().numpy(), scales.cpu().numpy()


# ------------------------------------------------------------- quantization


@pytest.mark.parametrize("m,k", [(1, 32), (3, 64), (5, 96), (1, 4096), (9, 4128), (333, 160)])
@pytest.mark.parametrize("t", [torch.float32, torch.float16, torch.bfloat16])
def test_quantize_random(bqm, m, k, t):
    rng = np.random.default_rng(m + k)
    x = torch.from_numpy((rng.standard_normal((m, k)) * np.exp2(rng.integers(-12, 12, (m, 1)))).astype(np.float32)).to(t)
    c, s = quantize(bqm, x.to(DEV))
    rc, rs = layer_ref.mxfp4_quantize(x.float().numpy())
    assert np.array_equal(s, rs) and np.array_equal(c, rc)


def test_quantize_every_midpoint_and_its_neighbours(bqm):
    """Each grid value and midpoint, one f32 step either side, both signs, at every block exponent."""
    at = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0], np.float32)
    v = np.concatenate([at, np.nextafter(at, np.float32(0)), np.nextafter(at, np.float32(9))])
    v = np.concatenate([v, -v, [-0.0, np.float32(7.9999995)]]).astype(np.float32)
    blocks = []
    for e in (-127, -126, -125, -120, -60, -1, 0, 1, 60, 120, 125):
        for top in (4.0, 7.75, 2.0):   # 2.0: the values above it set the exponent themselves
            for i in range(0, len(v), 31):
                b = np.zeros(32, np.float32)
                part = v[i:i + 31]
                b[:len(part)] = part
                b[31] = top
                blocks.append(np.ldexp(b.astype(np.float64), e).astype(np.float32))
    x = np.stack(blocks)
    c, s = quantize(bqm, dev(x))
    rc, rs = layer_ref.mxfp4_quantize(x)
    assert np.array_equal(s, rs) and np.array_equal(c, rc)


def test_quantize_all_bit_patterns(bqm):
    """Random f32 bit patterns (subnormals, infinities, NaN among them) and every bf16 pattern."""
    rng = np.random.default_rng(1)
    x = rng.integers(0, 1 << 32, (4096, 64), dtype=np.uint32).view(np.float32)
    small = rng.integers(0, 1 << 24, (64, 64), dtype=np.uint32).view(np.float32)     # zero, subnormal, smallest normal
    every = (np.arange(1 << 16, dtype=np.uint32) << 16).view(np.float32).reshape(-1, 64)
    zeros = np.zeros((2, 64), np.float32)
    zeros[1] = -0.0
    x = np.concatenate([x, small, every, zeros])
    c, s = quantize(bqm, dev(x))
    rc, rs = layer_ref.mxfp4_quantize(x)
    assert np.array_equal(s, rs) and np.array_equal(c, rc)


def test_quantize_strided_rows(bqm):
    rng = np.random.default_rng(2)
    wide = dev(rng.standard_normal((7, 200)).astype(np.float32))
    x = wide[:, 4:4 + 160]
    c, s = quantize(bqm, x)
    rc, rs = layer_ref.mxfp4_quantize(x.cpu().numpy())
    assert np.array_equal(s, rs) and np.array_equal(c, rc)


def test_dequantize_every_code_and_scale(bqm):
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))       # 512 values a row
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, axis=1)
    ref = layer_ref.mxfp4_values(codes, scales)
    y = bqm.bqm_mxfp4_dequantize(dev(codes), dev(scales)).cpu().numpy()
    with np.errstate(over="ignore"):
        want = ref.astype(np.float32)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(y), nan) and same_bits(y[~nan], want[~nan])
    for t in (torch.float16, torch.bfloat16):
        y = bqm.bqm_mxfp4_dequantize(dev(codes), dev(scales), t).cpu()
        w = torch.from_numpy(want).to(t)
        assert torch.equal(torch.isnan(y), torch.isnan(w))
        assert torch.equal(y.view(torch.int16)[~torch.isnan(w)], w.view(torch.int16)[~torch.isnan(w)])


# ----------------------------------------------------------------- products


def check(y, ref, T, factor, what):
    y = y.cpu().numpy().astype(np.float64)
    assert np.isfinite(y).all(), f"{what}: non-finite output"
    off = np.abs(y - ref)
    assert (off <= factor * T).all(), f"{what}: {np.max(off / np.maximum(T, 1e-300)):.3e} of sum|terms|, bound {factor:.3e}"


GEMM = [(1, 32, 1), (2, 64, 3), (17, 96, 33), (16, 4096, 96), (31, 160, 257), (128, 256, 256), (129, 512, 255),
        (300, 1056, 321), (64, 2880, 100), (512, 1024, 640), (5, 5120, 700), (33, 4096, 1000), (1, 17408, 40),
        (257, 288, 513), (65, 1024, 65), (1000, 128, 77)]


@pytest.mark.parametrize("m,k,n", GEMM)
def test_gemm_matches_64_bits(bqm, m, k, n):
    rng = np.random.default_rng(m + 3 * k + n)
    w, ws = random_mx(n, k, rng)
    xq, xs = random_mx(m, k, rng)
    y = torch.full((m, n), float("nan"), device=DEV)
    bqm.bqm_mxfp4_gemm(dev(w), dev(ws), dev(xq), dev(xs), y)
    ref, T = layer_ref.mxfp4_matmul(w, ws, layer_ref.mxfp4_values(xq, xs))
    check(y, ref, T, (3 * k / 64 + 2) * 2.0 ** -23, f"m={m} k={k} n={n}")


# More tokens than one workgroup takes, against few weight rows: chunks of tokens, with a short last one.
CHUNKS = [(65, 4096, 33), (98, 12512, 320), (63, 17088, 153), (130, 5120, 50), (200, 17408, 16), (129, 8192, 1), (257, 4128, 100),
          (33, 16384, 70), (96, 10240, 257), (513, 17408, 40)]


@pytest.mark.parametrize("m,k,n", CHUNKS)
def test_gemm_few_rows_of_long_k(bqm, m, k, n):
    rng = np.random.default_rng(m + 3 * k + n)
    w, ws = random_mx(n, k, rng)
    xq, xs = random_mx(m, k, rng)
    y = torch.full((m + 2, n), float("nan"), device=DEV)
    bqm.bqm_mxfp4_gemm(dev(w), dev(ws), dev(xq), dev(xs), y[1:m + 1])
    ref, T = layer_ref.mxfp4_matmul(w, ws, layer_ref.mxfp4_values(xq, xs))
    check(y[1:m + 1], ref, T, (3 * k / 64 + 2) * 2.0 ** -23, f"m={m} k={k} n={n}")
    assert bool(torch.isnan(y[0]).all()) and bool(torch.isnan(y[m + 1]).all())


@pytest.mark.parametrize("m,k,n", [(1, 512, 64), (40, 1024, 300), (300, 512, 300)])
def test_gemm_wide_scales(bqm, m, k, n):
    """Scales 80 binades apart."""
    rng = np.random.default_rng(m)
    w, ws = random_mx(n, k, rng, 87, 167)
    xq, xs = random_mx(m, k, rng, 87, 167)
    y = bqm.bqm_mxfp4_gemm(dev(w), dev(ws), dev(xq), dev(xs))
    ref, T = layer_ref.mxfp4_matmul(w, ws, layer_ref.mxfp4_values(xq, xs))
    check(y, ref, T, (3 * k / 64 + 2) * 2.0 ** -23, "wide scales")


@pytest.mark.parametrize("m", [1, 20, 200])
def test_gemm_one_hot_is_exact(bqm, m):
    """One nonzero activation per token: y is one product, bit for bit."""
    rng = np.random.default_rng(m)
    k, n = 1056, 130
    w, ws = random_mx(n, k, rng)
    at = rng.integers(0, k, m)
    xq = np.zeros((m, k // 2), np.uint8)
    xq[np.arange(m), at // 2] = 0x5 << (4 * (at % 2))               # 3.0
    xs = np.full((m, k // 32), 130, np.uint8)
    y = bqm.bqm_mxfp4_gemm(dev(w), dev(ws), dev(xq), dev(xs)).cpu().numpy()
    v = layer_ref.mxfp4_values(w, ws)
    assert np.array_equal(y, (24.0 * v[:, at].T).astype(np.float32))


@pytest.mark.parametrize("m", [1, 40, 200])
def test_gemm_nan_blocks_stay_in_their_row(bqm, m):
    rng = np.random.default_rng(7)
    k, n = 544, 70
    w, ws = random_mx(n, k, rng)
    xq, xs = random_mx(m, k, rng)
    ws[5, 3] = 255
    xs[m - 1, 16] = 255
    y = bqm.bqm_mxfp4_gemm(dev(w), dev(ws), dev(xq), dev(xs)).cpu().numpy()
    want = np.zeros((m, n), bool)
    want[:, 5] = True
    want[m - 1] = True
    assert np.array_equal(np.isnan(y), want)


GEMV = [(1, 32, 1), (1, 4096, 1000), (2, 1280, 333), (3, 96, 17), (4, 5120, 64), (5, 4096, 257), (6, 4096, 257),
        (7, 1056, 100), (9, 4096, 129), (10, 544, 77), (11, 2880, 50), (16, 4096, 96), (16, 32, 16), (1, 17408, 333),
        (9, 17408, 40), (16, 8224, 33), (1, 512, 70000), (2, 2048, 4096), (1, 17408, 9000), (2, 9728, 8200),
        (5, 4096, 8300), (3, 1536, 9001), (4, 64, 9000)]


@pytest.mark.parametrize("m,k,n", GEMV)
def test_gemv_matches_64_bits(bqm, m, k, n):
    rng = np.random.default_rng(m + 5 * k + n)
    w, ws = random_mx(n, k, rng)
    x = rng.standard_normal((m, k)).astype(np.float32)
    x *= np.where(rng.random((m, k)) < 0.01, 10, 1).astype(np.float32)
    y = torch.full((m, n), float("nan"), device=DEV)
    bqm.bqm_mxfp4_gemv(dev(w), dev(ws), dev(x), y)
    ref, T = layer_ref.mxfp4_matmul(w, ws, x.astype(np.float64))
    check(y, ref, T, (8 * 16 + -(-k // 512) + 4) * 2.0 ** -23, f"m={m} k={k} n={n}")


@pytest.mark.parametrize("k,n", [(4096, 500), (1056, 100), (17408, 50), (512, 9000)])
def test_gemv_token_does_not_depend_on_m(bqm, k, n):
    rng = np.random.default_rng(k)
    w, ws = (dev(a) for a in random_mx(n, k, rng))
    x = dev(rng.standard_normal((16, k)).astype(np.float32))
    one = torch.cat([bqm.bqm_mxfp4_gemv(w, ws, x[t:t + 1]) for t in range(16)])
    for m in range(2, 17):
        assert torch.equal(bqm.bqm_mxfp4_gemv(w, ws, x[:m]), one[:m]), m


def test_gemv_wide_activations_and_one_hot(bqm):
    """Activations 32 binades apart keep their 24 bits; one nonzero value gives one exact product."""
    rng = np.random.default_rng(3)
    k, n, m = 2080, 200, 9
    w, ws = random_mx(n, k, rng)
    x = (rng.standard_normal((m, k)) * np.exp2(rng.uniform(-16, 16, (m, k)))).astype(np.float32)
    y = bqm.bqm_mxfp4_gemv(dev(w), dev(ws), dev(x))
    ref, T = layer_ref.mxfp4_matmul(w, ws, x.astype(np.float64))
    check(y, ref, T, (8 * 16 + 5 + 4) * 2.0 ** -23, "wide activations")
    at = rng.integers(0, k, m)
    hot = np.zeros((m, k), np.float32)
    hot[np.arange(m), at] = np.float32(-1.2345678)
    y = bqm.bqm_mxfp4_gemv(dev(w), dev(ws), dev(hot)).cpu().numpy()
    ref = np.float64(np.float32(-1.2345678)) * layer_ref.mxfp4_values(w, ws)[:, at].T
    assert np.array_equal(y, ref.astype(np.float32))


def test_gemv_special_values_stay_in_their_row(bqm):
    rng = np.random.default_rng(4)
    k, n, m = 1024, 40, 7
    w, ws = random_mx(n, k, rng)
    w |= 0x22                                        # no zero codes: an infinity times any of them is not finite
    ws[3, 8] = 255
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[2, 9] = np.nan
    x[5, 1000] = np.inf
    x[0] = 0
    y = bqm.bqm_mxfp4_gemv(dev(w), dev(ws), dev(x)).cpu().numpy()
    bad = np.zeros((m, n), bool)
    bad[:, 3] = bad[2] = bad[5] = True
    assert np.array_equal(~np.isfinite(y), bad)
    assert np.isnan(y[:, 3]).all() and np.isnan(y[2]).all()
    assert (y[0][~bad[0]] == 0).all()


def test_products_agree_on_quantized_activations(bqm):
    """The decode product of the dequantized activations is the GEMM's, up to both bounds."""
    rng = np.random.default_rng(6)
    k, n, m = 4096, 300, 16
    w, ws = (dev(a) for a in random_mx(n, k, rng))
    x = dev(rng.standard_normal((m, k)).astype(np.float32))
    xq, xs = bqm.bqm_mxfp4_quantize(x)
    back = bqm.bqm_mxfp4_dequantize(xq, xs)
    a, b = bqm.bqm_mxfp4_gemm(w, ws, xq, xs), bqm.bqm_mxfp4_gemv(w, ws, back)
    T = layer_ref.mxfp4_matmul(w.cpu().numpy(), ws.cpu().numpy(), back.cpu().numpy().astype(np.float64))[1]
    off = (a - b).abs().cpu().numpy()
    assert (off <= ((3 * k / 64 + 2) + (8 * 16 + 12)) * 2.0 ** -23 * T).all()


def test_products_of_unaligned_scales_and_streams(bqm):
    """Scale tensors at odd addresses, on a stream of their own."""
    rng = np.random.default_rng(8)
    k, n, m = 1024, 130, 12
    w, ws = random_mx(n, k, rng)
    xq, xs = random_mx(m, k, rng)
    x = rng.standard_normal((m, k)).astype(np.float32)

    def odd(a):
        flat = torch.zeros(a.size + 1, dtype=torch.uint8, device=DEV)
        flat[1:] = dev(a).view(-1)
        return flat[1:].view(a.shape)

    args = dev(w), dev(ws), dev(xq), dev(xs), dev(x)
    want = bqm.bqm_mxfp4_gemm(*args[:4]), bqm.bqm_mxfp4_gemv(args[0], args[1], args[4])
    so = odd(ws), odd(xs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = bqm.bqm_mxfp4_gemm(args[0], so[0], args[2], so[1]), bqm.bqm_mxfp4_gemv(args[0], so[0], args[4])
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals(bqm):
    u8 = dict(dtype=torch.uint8, device=DEV)
    w, ws = torch.zeros((8, 32), **u8), torch.zeros((8, 2), **u8)
    x = torch.zeros((4, 64), device=DEV)
    with pytest.raises(ValueError):
        bqm.bqm_mxfp4_gemv(w, ws[:, :1].contiguous(), x)
    with pytest.raises(ValueError):
        bqm.bqm_mxfp4_gemv(w, ws, x.half())
    with pytest.raises(ValueError):
        bqm.bqm_mxfp4_gemm(w, ws, w[:, :16].contiguous(), ws)
    with pytest.raises(bqm.BqmError):
        bqm.bqm_mxfp4_gemv(w, ws, torch.zeros((17, 64), device=DEV))
    with pytest.raises(bqm.BqmError):
        bqm.bqm_mxfp4_quantize(torch.zeros((4, 48), device=DEV))
    with pytest.raises(bqm.BqmError):
        bqm.bqm_mxfp4_quantize(torch.zeros((4, 65), device=DEV)[:, :64])    # rows not 16-byte aligned
    with pytest.raises(ValueError):
        bqm.bqm_mxfp4_quantize(torch.zeros((4, 64), dtype=torch.int32, device=DEV))
