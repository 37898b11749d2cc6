"""Plain 64-bit implementations of the operators in include/bqmm_layer.h, for the tests (numpy, host arrays)."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def rmsnorm(x, res, gain, eps):
    """(y, s): the norm of s = x + res and s itself, in 64 bits."""
    s = x.astype(np.float64)
    if res is not None:
        s = s + res.astype(np.float64)
    y = s / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return (y if gain is None else y * gain.astype(np.float64)), s


def mxfp4_quantize(x):
    """(codes, scales) of f32 values x [m, k]: the nearest of the 15 values, ties to the even code."""
    m, k = x.shape
    b = x.astype(np.float64).reshape(m, k // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(axis=2))
    _, e = np.frexp(amax)                       # amax = f * 2^e, 0.5 <= f < 1
    s = np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    v = np.abs(b) * np.exp2(127.0 - s)[:, :, None]
    code = np.zeros(v.shape, np.int64)
    grid = E2M1[:8]
    for i in range(7):
        mid = (grid[i] + grid[i + 1]) / 2
        # past the midpoint, or on it with an odd code below
        code += (v > mid) | ((v == mid) & (i % 2 == 1))
    code = np.where(np.signbit(b), code + 8, code)
    code = np.where(bad[:, :, None], 0, code).reshape(m, k).astype(np.uint8)
    s = np.where(bad, 255, s).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), s


def mxfp4_values(codes, scales):
    """The values of MXFP4 codes [m, k/2] and scales [m, k/32], in 64 bits."""
    m, half = codes.shape
    v = np.empty((m, 2 * half))
    v[:, 0::2] = E2M1[codes & 15]
    v[:, 1::2] = E2M1[codes >> 4]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return v * np.repeat(s, 32, axis=1)


def mxfp4_matmul(w, ws, x):
    """(x . W^T, sum |terms|) for 64-bit x [m, k] and MXFP4 weights."""
    v = mxfp4_values(w, ws)
    return x @ v.T, np.abs(x) @ np.abs(v).T


def logprobs(l, tokens, top):
    """(logp, lse, entropy, ids, top_logp) of 64-bit logits [m, n]; -inf rows and NaN rows as the header says."""
    m, n = l.shape
    bad = np.isnan(l).any(axis=1) | (l == np.inf).any(axis=1)
    safe = np.where(bad[:, None], 0.0, l)
    big = safe.max(axis=1, keepdims=True)
    empty = np.isneginf(big[:, 0])
    big = np.where(np.isneginf(big), 0.0, big)
    d = safe - big
    e = np.exp(d)
    z = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        logz = np.log(z)
        lse = np.where(empty, -np.inf, (big + logz)[:, 0])
        ent = np.where(empty, 0.0, (logz - np.where(e > 0, e * np.where(e > 0, d, 0.0), 0.0).sum(axis=1, keepdims=True) / z)[:, 0])
        all_logp = np.where(empty[:, None], -np.inf, d - logz)
    lse[bad] = np.nan
    ent[bad] = np.nan
    all_logp[bad] = np.nan
    logp = np.full(tokens.shape, np.nan)
    for t in range(m):
        for i in range(tokens.shape[1]):
            if 0 <= tokens[t, i] < n:
                logp[t, i] = all_logp[t, tokens[t, i]]
    # a NaN is below -inf; equal values by column
    ids = np.empty((m, top), np.int64)
    for t in range(m):
        rank = np.where(np.isnan(l[t]), -np.inf, l[t])
        ids[t] = np.lexsort((np.arange(n), -rank, np.isnan(l[t])))[:top]
    return logp, lse, ent, ids, np.take_along_axis(all_logp, ids, axis=1)
