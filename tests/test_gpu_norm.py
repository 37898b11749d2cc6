"""RMS norm with residual and its 8-bit outputs, against 64 bits and against the library's quantizers.

Tolerance of an f32 y, u = 2^-24: s is one rounding (u); the sum of squares is
a chain of c fma per thread (at most 16, or 8 * ceil(k / 8192) for rows longer
than 16384), 6 steps over the wave and at most 16 over the workgroup, on
squares that are 2u off: (c + 24) u, halved by the root; division by k, eps,
root, reciprocal and two products add at most 6u.  In all (c / 2 + 19) u of
|y|; a 16-bit y adds its own half ulp.
"""
import numpy as np
import pytest

import layer_ref
import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
EPS = 1e-6


@pytest.fixture(scope="module")
def bqm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_matmul_02_amd as m

    m.lib()
    return m


def inputs(m, k, t, seed, ld=None, offset=0):
    """x, res (rows ld apart, starting `offset` elements into their storage) and gain on the GPU."""
    g = torch.Generator().manual_seed(seed)
    ld = ld or k

    def one(std):
        flat = torch.zeros(offset + m * ld, dtype=t)
        v = flat[offset:].view(m, ld)[:, :k]
        v.copy_((torch.randn((m, k), generator=g) * std).to(t))
        dev = flat.to(DEV)
        return dev[offset:].view(m, ld)[:, :k]

    return one(1.0), one(3.0), (1.0 + 0.1 * torch.randn(k, generator=g)).to(DEV)


def bound(k, t):
    chain = max(16, 8 * -(-k // 8192))
    return (chain / 2 + 19) * 2.0 ** -24 + HALF_ULP[t]


def host(t):
    return t.detach().float().cpu().numpy()


def check(y, ref, k, t, what):
    got = host(y).astype(np.float64)
    assert np.isfinite(got).all(), what
    # 2^-25: half the smallest fp16 step, for subnormal results
    off = np.abs(got - ref) - bound(k, t) * np.abs(ref) - (2.0 ** -25 if t == torch.float16 else 0.0)
    assert off.max() <= 0, f"{what}: {off.max():.3e} beyond the bound"


SIZES = [(1, 1), (3, 2), (2, 31), (5, 64), (1, 255), (7, 1024), (4, 1025), (1, 4096), (9, 4100), (3, 5120), (2, 8191),
         (2, 16384), (2, 16385), (3, 20480), (1, 50000)]


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", SIZES)
def test_norm_matches_64_bits(bqm, m, k, t):
    dt = TYPES[t]
    x, res, gain = inputs(m, k, dt, 10 * m + k)
    for r, g in ((res, gain), (None, gain), (res, None), (None, None)):
        ref, s = layer_ref.rmsnorm(host(x), None if r is None else host(r), None if g is None else host(g), EPS)
        for out in {torch.float32, dt}:
            y = torch.full((m, k), float("nan"), dtype=out, device=DEV)
            h = None if r is None else torch.full((m, k), float("nan"), dtype=dt, device=DEV)
            y, h = bqm.bqm_add_rmsnorm(x, r, g, EPS, h=h, y=y)
            check(y, ref, k, out, f"{t} {m}x{k} res={r is not None} gain={g is not None}")
            if r is not None:
                assert torch.equal(h, (x.float() + r.float()).to(dt))


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("m,k,ld,offset", [(5, 63, 64, 0), (5, 64, 67, 0), (5, 64, 64, 1), (3, 4096, 4104, 0),
                                           (3, 4096, 4097, 3), (2, 20000, 20003, 5)])
def test_strides_and_alignment_change_nothing(bqm, m, k, ld, offset, t):
    """The same values in dense, aligned rows give the same bits."""
    x, res, gain = inputs(m, k, TYPES[t], 77 + k, ld, offset)
    y, h = bqm.bqm_add_rmsnorm(x, res, gain, EPS)
    yd, hd = bqm.bqm_add_rmsnorm(x.contiguous(), res.contiguous(), gain, EPS)
    assert torch.equal(y, yd) and torch.equal(h, hd)


@pytest.mark.parametrize("k", [64, 1000, 4096, 20480])
def test_rows_do_not_depend_on_each_other(bqm, k):
    x, res, gain = inputs(37, k, torch.float32, 5)
    y, _ = bqm.bqm_add_rmsnorm(x, res, gain, EPS)
    for t in (0, 17, 36):
        one, _ = bqm.bqm_add_rmsnorm(x[t:t + 1], res[t:t + 1], gain, EPS)
        assert torch.equal(one[0], y[t])


@pytest.mark.parametrize("k", [96, 4096, 16416])
def test_residual_in_place(bqm, k):
    for which in (0, 1):
        x, res, gain = inputs(6, k, torch.bfloat16, 9)
        want_y, want_h = bqm.bqm_add_rmsnorm(x, res, gain, EPS)
        h = (x, res)[which]
        y, h2 = bqm.bqm_add_rmsnorm(x, res, gain, EPS, h=h)
        assert h2.data_ptr() == h.data_ptr()
        assert torch.equal(y, want_y) and torch.equal(h, want_h)


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", [(1, 32), (3, 96), (2, 1024), (5, 1056), (1, 4096), (9, 5120), (2, 16416)])
def test_q8_1_output(bqm, m, k, t):
    """Bit for bit the quantizer's output on the f32 norm, and the oracle's."""
    x, res, gain = inputs(m, k, TYPES[t], 100 + k)
    y, h = bqm.bqm_add_rmsnorm(x, res, gain, EPS)
    xq, xds, h2 = bqm.bqm_add_rmsnorm_q8_1(x, res, gain, EPS, xq=torch.full((m, k), 99, dtype=torch.int8, device=DEV),
                                           xds=torch.full((m, k // 32, 2), float("nan"), device=DEV))
    q, ds = oracle.q8_1_quantize(host(y))
    assert torch.equal(h, h2)
    assert np.array_equal(xq.cpu().numpy(), q) and np.array_equal(xds.cpu().numpy(), ds)
    q2, ds2 = bqm.bqm_q8_1_quantize(y)
    assert torch.equal(xq, q2) and torch.equal(xds, ds2)


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", [(1, 16), (3, 112), (2, 144), (2, 1024), (5, 1040), (1, 4096), (9, 5120), (2, 16400)])
def test_e4m3_output(bqm, m, k, t):
    x, res, gain = inputs(m, k, TYPES[t], 200 + k)
    y, h = bqm.bqm_add_rmsnorm(x, res, gain, EPS)
    xq, xs, h2 = bqm.bqm_add_rmsnorm_e4m3_blk(x, res, gain, EPS,
                                              xq=torch.full((m, k), 99, dtype=torch.uint8, device=DEV),
                                              xs=torch.full((m, (k + 127) // 128), float("nan"), device=DEV))
    q, s = oracle.e4m3_blk_quantize(host(y))
    assert torch.equal(h, h2)
    assert np.array_equal(xq.cpu().numpy(), q) and np.array_equal(xs.cpu().numpy(), s)


def test_8_bit_outputs_of_strided_rows(bqm):
    x, res, gain = inputs(4, 1024, torch.bfloat16, 3, ld=1027, offset=1)
    y, _ = bqm.bqm_add_rmsnorm(x, res, gain, EPS)
    xq, xds, _ = bqm.bqm_add_rmsnorm_q8_1(x, res, gain, EPS)
    q2, ds2 = bqm.bqm_q8_1_quantize(y)
    assert torch.equal(xq, q2) and torch.equal(xds, ds2)
    eq, es, _ = bqm.bqm_add_rmsnorm_e4m3_blk(x, res, gain, EPS)
    q3, s3 = bqm.bqm_e4m3_blk_quantize(y)
    assert torch.equal(eq, q3) and torch.equal(es, s3)


@pytest.mark.parametrize("k", [64, 4096, 20480])
def test_zero_rows_and_special_values(bqm, k):
    x = torch.zeros((6, k), device=DEV)
    x[1, k // 2] = 3.0
    x[2] = 1e-30                       # squares underflow: eps decides
    x[3, 5] = float("inf")
    x[4, 7] = float("nan")
    x[5] = 1e15
    y, _ = bqm.bqm_add_rmsnorm(x, None, None, EPS)
    y = y.cpu().numpy()
    assert (y[0] == 0).all()
    ref, _ = layer_ref.rmsnorm(host(x[[1, 2, 5]]), None, None, EPS)
    for got, want in zip(y[[1, 2, 5]], ref):
        assert np.allclose(got, want, rtol=bound(k, torch.float32), atol=0)
    assert np.isnan(y[3, 5]) and (np.delete(y[3], 5) == 0).all()   # inf / inf, and the rest by an infinite root
    assert np.isnan(y[4]).all()
    xq, xds, _ = bqm.bqm_add_rmsnorm_q8_1(x[:1], None, None, EPS)
    assert (xq == 0).all() and (xds == 0).all()
    y, _ = bqm.bqm_add_rmsnorm(x[:1], None, None, 0.0)
    assert torch.isnan(y).all()        # 0 * 1/sqrt(0)


def test_many_rows_and_another_stream(bqm):
    """More rows than one launch has workgroups for, on a stream of their own."""
    m, k = (1 << 22) + 5, 8
    s = torch.cuda.Stream()
    x = torch.randn((m, k), device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, _ = bqm.bqm_add_rmsnorm(x, None, None, EPS)
    s.synchronize()
    d = x.double()
    ref = d / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    assert ((y.double() - ref).abs() <= bound(k, torch.float32) * ref.abs()).all()


def test_refusals(bqm):
    x = torch.zeros((4, 64), device=DEV)
    with pytest.raises(ValueError):
        bqm.bqm_add_rmsnorm(x, None, None, EPS, h=x)                      # h without res
    with pytest.raises(ValueError):
        bqm.bqm_add_rmsnorm(x, x.half(), None, EPS)                       # another type
    with pytest.raises(ValueError):
        bqm.bqm_add_rmsnorm(x, x[:2], None, EPS)                          # another shape
    with pytest.raises(ValueError):
        bqm.bqm_add_rmsnorm(x.t(), None, None, EPS)                       # columns
    with pytest.raises(ValueError):
        bqm.bqm_add_rmsnorm(x, None, torch.ones(63, device=DEV), EPS)
    with pytest.raises(ValueError):
        bqm.bqm_add_rmsnorm(x.cpu(), None, None, EPS)
    with pytest.raises(ValueError):
        bqm.bqm_add_rmsnorm(x.double(), None, None, EPS)
    with pytest.raises(bqm.BqmError):
        bqm.bqm_add_rmsnorm(x, None, None, -1.0)
    with pytest.raises(bqm.BqmError):
        bqm.bqm_add_rmsnorm(x, None, None, EPS, out_dtype=torch.float16)  # neither f32 nor x's
    with pytest.raises(bqm.BqmError):
        bqm.bqm_add_rmsnorm_q8_1(x[:, :48], None, None, EPS)
    with pytest.raises(bqm.BqmError):
        bqm.bqm_add_rmsnorm_e4m3_blk(x[:, :24], None, None, EPS)
