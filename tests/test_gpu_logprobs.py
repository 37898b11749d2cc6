"""Log probabilities, log-sum-exp, entropy and top alternatives against 64 bits.

Tolerance: with u = 2^-24, a term e^(l-m) is off by at most (4 |l - m| + 4) u
of itself (the difference and its product with log2 e rounded, the exponential
to 1 ulp); the terms' mean of |l - m| under p is H + log Z - ... <= log n; a
thread adds c <= 16 ceil(n / 4096) terms one by one and the joins take 16 more
steps.  So Z and S / Z are off by at most D = (4 log n + c + 24) 2u relative to
1 + log n, lse by that and its own rounding, and log p by that and the
rounding of l - m.  Ids are exact.
"""
import math

import numpy as np
import pytest

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


def call(bqm, logits, tokens, top):
    m = logits.shape[0]
    t = 0 if tokens is None else tokens.shape[1]
    nan = float("nan")
    out = (torch.full((m, t), nan, device=DEV), torch.full((m,), nan, device=DEV), torch.full((m,), nan, device=DEV),
           torch.full((m, top), -7, dtype=torch.int32, device=DEV), torch.full((m, top), nan, device=DEV))
    size = bqm.bqm_logprobs_workspace(m, logits.shape[1], top)
    workspace = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) if size else None   # needs no contents
    got = bqm.bqm_logprobs(logits, tokens, top, out=out, workspace=workspace)
    return [v.cpu().numpy() for v in got]


def near(got, ref, tol, what):
    got = got.astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN"
    assert np.array_equal(np.isinf(got), np.isinf(ref)), f"{what}: infinities"
    ok = np.isfinite(ref)
    assert (got[~ok & ~np.isnan(ref)] == ref[~ok & ~np.isnan(ref)]).all(), what
    tol = np.broadcast_to(tol, ref.shape)
    assert (np.abs(got - ref)[ok] <= tol[ok]).all(), f"{what}: {np.max(np.abs(got - ref)[ok] / tol[ok]):.3f} of the bound"


def check(bqm, logits, tokens, top, what=""):
    l = logits.float().cpu().numpy().astype(np.float64)
    m, n = l.shape
    tok = np.zeros((m, 0), np.int32) if tokens is None else tokens.cpu().numpy()
    logp, lse, ent, ids, top_logp = call(bqm, logits, tokens, top)
    r = layer_ref.logprobs(l, tok, top)
    u = 2.0 ** -24
    ln = math.log(n) + 1
    base = (4 * ln + 16 * -(-n // 4096) + 24) * 2 * u * (1 + ln)
    near(lse, r[1], base + 4 * u * np.abs(np.where(np.isfinite(r[1]), r[1], 0)), what + " lse")
    near(ent, r[2], base, what + " entropy")
    big = np.abs(l[np.isfinite(l)]).max() if np.isfinite(l).any() else 0.0
    for g, w, name in ((logp, r[0], " logp"), (top_logp, r[4], " top_logp")):
        near(g, w, base + 4 * u * (2 * big + np.abs(np.where(np.isfinite(w), w, 0))), what + name)
    assert np.array_equal(ids, r[3]), f"{what}: ids"


def normal(m, n, seed, t=torch.float32, std=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((m, n), generator=g) * std).to(t).to(DEV)


def some_tokens(m, n, t, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, n, (m, t), generator=g, dtype=torch.int32).to(DEV)


SIZES = [(1, 1), (1, 2), (3, 5), (2, 63), (2, 64), (2, 65), (3, 1000), (1, 4095), (2, 4096), (2, 4097), (5, 20000),
         (1, 64448), (4, 131071), (1, 262144), (600, 3000), (3000, 300), (2100, 5000)]


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n", SIZES)
def test_matches_64_bits(bqm, m, n, t):
    logits = normal(m, n, m + n, TYPES[t])
    check(bqm, logits, some_tokens(m, n, 2, 1), min(n, 20), f"{t} {m}x{n}")


@pytest.mark.parametrize("top", [0, 1, 2, 5, 31, 32])
@pytest.mark.parametrize("m,n", [(1, 32), (1, 100000), (2, 9000), (2500, 64)])
def test_every_top_and_token_count(bqm, m, n, top):
    logits = normal(m, n, 7 * top + n)
    for t in (0, 1, 70):
        check(bqm, logits, some_tokens(m, n, t, top) if t else None, top, f"{m}x{n} top {top} tokens {t}")


@pytest.mark.parametrize("m", [1, 3, 2500])
def test_rows_any_stride_and_alignment(bqm, m):
    for n, ld, offset in ((5000, 5001, 1), (5000, 5003, 2), (4999, 5016, 3)):
        for t in (torch.float32, torch.bfloat16):
            flat = normal(1, offset + m * ld, ld, t)[0]
            rows = flat[offset:].view(m, ld)[:, :n]
            check(bqm, rows[:4], some_tokens(min(m, 4), n, 1, 3), 7, f"ld {ld} offset {offset}")
            if m > 4:
                got = call(bqm, rows, None, 7)
                want = call(bqm, rows.contiguous(), None, 7)
                assert np.array_equal(got[3], want[3])
                assert np.allclose(got[1], want[1], rtol=1e-5)


@pytest.mark.parametrize("m,n", [(1, 70000), (4, 9001), (2200, 500)])
def test_order_of_the_logits(bqm, m, n):
    """Rising, falling, constant, few distinct and saw-toothed rows: the bounds' worst cases and ties."""
    i = torch.arange(n, dtype=torch.float32)
    for name, row in (("rising", i / n * 9), ("falling", -i / n * 9), ("constant", torch.full((n,), 1.5)),
                      ("two values", (i.long() * 7919 % 11 == 3).float()), ("saw", (i % 4096) / 300),
                      ("signed zeros", torch.where(i.long() % 2 == 0, 0.0, -0.0)),
                      ("blocks", torch.div(i, 16, rounding_mode="floor") % 64)):
        logits = row.expand(min(m, 4), n).contiguous().to(DEV)
        check(bqm, logits, None, 32, name)
        if m > 4:
            ids = call(bqm, row.expand(m, n).contiguous().to(DEV), None, 32)[3]
            assert (ids == ids[0]).all(), name


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [50, 5000, 70000])
def test_masks(bqm, n, t):
    """Masks of -inf and of the type's lowest value, rows with one token or none left, NaN and infinities."""
    dt = TYPES[t]
    logits = normal(12, n, n, dt)
    low = torch.finfo(dt).min
    logits[0, 1:] = -math.inf            # one left
    logits[1] = -math.inf                # none left
    logits[2] = low                      # all at the lowest value
    logits[3, n // 2:] = low
    logits[4, : n - 3] = -math.inf       # fewer than top_k left
    logits[5, ::2] = -math.inf
    logits[6, n // 3] = math.nan
    logits[7, n - 1] = math.inf
    logits[8] = math.nan
    logits[9, 0] = -math.inf
    logits[10] = -math.inf
    logits[10, n - 1] = low
    logits[11, 2:] = math.nan
    tokens = torch.tensor([[0, 1, n - 1, -1, n]] * 12, dtype=torch.int32, device=DEV)
    check(bqm, logits, tokens, 20, f"masks {t} {n}")


def test_padding_tokens_read_nothing(bqm):
    logits = normal(2, 100, 0)
    tokens = torch.tensor([[-1, -100, 2 ** 31 - 1], [-2 ** 31, 100, 99]], dtype=torch.int32, device=DEV)
    logp = call(bqm, logits, tokens, 0)[0]
    assert np.isnan(logp.reshape(-1)[:5]).all() and np.isfinite(logp[1, 2])


def test_two_streams_and_default_outputs(bqm):
    a, b = normal(2, 70000, 1), normal(2, 70000, 2)
    want = [bqm.bqm_logprobs(v, None, 8) for v in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, v in zip(streams, (a, b)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(bqm.bqm_logprobs(v, None, 8))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))


def test_refusals(bqm):
    logits = torch.zeros((2, 10), device=DEV)
    with pytest.raises(bqm.BqmError):
        bqm.bqm_logprobs(logits, None, 11)
    with pytest.raises(bqm.BqmError):
        bqm.bqm_logprobs(torch.zeros((2, 100), device=DEV), None, 33)
    with pytest.raises(bqm.BqmError):
        bqm.bqm_logprobs(logits, None, -1)
    with pytest.raises(ValueError):
        bqm.bqm_logprobs(logits, torch.zeros((2, 1), dtype=torch.int64, device=DEV), 0)
    with pytest.raises(ValueError):
        bqm.bqm_logprobs(logits, torch.zeros((3, 1), dtype=torch.int32, device=DEV), 0)
    with pytest.raises(ValueError):
        bqm.bqm_logprobs(logits.t(), None, 0)
    with pytest.raises(ValueError):
        bqm.bqm_logprobs(logits.double(), None, 0)
    with pytest.raises(ValueError):
        bqm.bqm_logprobs(torch.zeros((1, 70000), device=DEV), None, 1, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))
