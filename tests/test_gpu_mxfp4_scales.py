"""The MXFP4 products over the whole range of scale bytes, one nonzero activation per token, so that every output is
one product: exact up to the one rounding of the result."""
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


def every_scale(k, last, seed):
    """Weights of random codes, row r at scale byte r throughout: 0 .. last."""
    rng = np.random.default_rng(seed)
    n = last + 1
    return rng.integers(0, 256, (n, k // 2)).astype(np.uint8), np.repeat(np.arange(n, dtype=np.uint8)[:, None], k // 32, axis=1)


def one_hot(m, k, value, seed):
    at = np.random.default_rng(seed).integers(0, k, m)
    x = np.zeros((m, k), np.float32)
    x[np.arange(m), at] = value
    return x, at


# up to five tokens and more are kernels of their own; k % 128 != 0 and k > 4096 are variants
@pytest.mark.parametrize("m,k", [(1, 512), (4, 1056), (5, 4608), (7, 512), (11, 1056), (16, 4608)])
@pytest.mark.parametrize("e", [100, 27, 0, -60, -100])
def test_gemv_every_scale(bqm, m, k, e):
    w, ws = every_scale(k, 252, m + k)
    x, at = one_hot(m, k, np.ldexp(np.float32(-1.2345678), e), m)
    y = bqm.bqm_mxfp4_gemv(dev(w), dev(ws), dev(x)).cpu().numpy()
    ref = x[np.arange(m), at].astype(np.float64)[:, None] * layer_ref.mxfp4_values(w, ws)[:, at].T
    normal = (np.abs(ref) >= 2.0 ** -126) & (np.abs(ref) < 2.0 ** 127) | (ref == 0)
    rows = normal.all(axis=0)
    assert rows.sum() >= 250 - abs(e) - 5
    # products whose three parts are normal too: 16 bits above the smallest normal number
    whole = rows & (np.abs(np.where(ref == 0, 1.0, ref)) >= 2.0 ** -108).all(axis=0)
    assert np.array_equal(y[:, whole], ref[:, whole].astype(np.float32))
    # below, what the second and third part lose where their products are subnormal
    assert (np.abs(y[:, rows] - ref[:, rows]) <= 2.0 ** -125 + 2.0 ** -24 * np.abs(ref[:, rows])).all()


@pytest.mark.parametrize("m,k", [(1, 512), (16, 1056)])
def test_gemv_of_tiny_blocks(bqm, m, k):
    """Weights that the quantizer stores at scale 0 (zeros, subnormals and their neighbours), made visible by a large x."""
    rng = np.random.default_rng(k)
    full = (rng.integers(-12, 13, (40, k)) * 2.0 ** -128).astype(np.float32)
    full[3] = 0
    w, ws = (v for v in bqm.bqm_mxfp4_quantize(dev(full)))
    assert int(ws.max()) <= 2 and int(ws[3].max()) == 0
    x, at = one_hot(m, k, np.float32(2.0 ** 100), 1)
    y = bqm.bqm_mxfp4_gemv(w, ws, dev(x)).cpu().numpy()
    ref = 2.0 ** 100 * layer_ref.mxfp4_values(w.cpu().numpy(), ws.cpu().numpy())[:, at].T
    assert np.count_nonzero(ref) and np.array_equal(y, ref.astype(np.float32))


@pytest.mark.parametrize("m,k", [(1, 512), (16, 1056)])
def test_gemv_of_tiny_activations(bqm, m, k):
    """Bits of x below 2^-133 are lost, those above are not."""
    w, ws = every_scale(k, 252, m + k)
    for e in (-112, -118, -126, -130, -133):
        x, at = one_hot(m, k, np.ldexp(1.2345678, e).astype(np.float32), m)
        y = bqm.bqm_mxfp4_gemv(dev(w), dev(ws), dev(x)).cpu().numpy()[:, 200:]
        v = layer_ref.mxfp4_values(w, ws)[200:, at].T
        ref = x[np.arange(m), at].astype(np.float64)[:, None] * v
        assert (np.abs(y - ref) <= np.abs(v) * 2.0 ** -133 + 2.0 ** -24 * np.abs(ref)).all(), e


# few tokens and tiles; scale rows aligned to 16 bytes and not
@pytest.mark.parametrize("m,k", [(1, 512), (20, 1056), (200, 512), (200, 1056), (700, 512)])
@pytest.mark.parametrize("total", [254, 200, 160, 330])
def test_gemm_scales_that_meet_their_opposite(bqm, m, k, total):
    """A small scale on one side and a large one on the other: byte pairs of one sum, over all bytes."""
    rng = np.random.default_rng(m + k)
    n = 255
    w, ws = every_scale(k, n - 1, m)
    at = rng.integers(0, k, m)
    for block in range(0, n, 85):
        # tokens at scale total - s meet row s
        s = min(max(total - block, 0), 254)
        xq = np.zeros((m, k // 2), np.uint8)
        xq[np.arange(m), at // 2] = 0xD << (4 * (at % 2))               # -3.0
        xs = np.full((m, k // 32), s, np.uint8)
        y = bqm.bqm_mxfp4_gemm(dev(w), dev(ws), dev(xq), dev(xs)).cpu().numpy()
        ref = -3.0 * 2.0 ** (s - 127.0) * layer_ref.mxfp4_values(w, ws)[:, at].T
        rows = ((np.abs(ref) >= 2.0 ** -126) & (np.abs(ref) < 2.0 ** 127) | (ref == 0)).all(axis=0)
        assert rows.sum() > 40
        assert np.array_equal(y[:, rows], ref[:, rows].astype(np.float32)), f"scale {s}"


@pytest.mark.parametrize("m,k", [(1, 512), (20, 1056), (700, 512)])
def test_gemm_past_the_range(bqm, m, k):
    """Products past f32's range are infinite with their sign, those inside it whole, and zero codes stay zero."""
    w, ws = every_scale(k, 254, m)
    at = np.random.default_rng(m).integers(0, k, m)
    xq = np.zeros((m, k // 2), np.uint8)
    xq[np.arange(m), at // 2] = 0x2 << (4 * (at % 2))                   # 1.0
    xs = np.full((m, k // 32), 254, np.uint8)                           # times 2^127
    y = bqm.bqm_mxfp4_gemm(dev(w), dev(ws), dev(xq), dev(xs)).cpu().numpy()
    ref = 2.0 ** 127 * layer_ref.mxfp4_values(w, ws)[:, at].T
    with np.errstate(over="ignore"):
        want = ref.astype(np.float32)
    assert np.isinf(want).any() and np.isfinite(want[ref != 0]).any()
    assert np.array_equal(y, want)
