"""Plain 64-bit implementations of the operators in include/bqmm_groups.h, for the tests (numpy, host arrays)."""
import numpy as np

import layer_ref


def route(l, top, renorm):
    """(ids, weights, the weights' error in steps of 2^-24 relative) of 64-bit logits [m, e].

    The error counts, for an f32 evaluation: the difference to the largest (half a step of it, so |d| steps of the
    exponential), six for the exponential, a sum of at most 22 dependent additions, and the division.
    """
    m, e = l.shape
    ids = np.full((m, top), -1)
    weights, steps = np.zeros((m, top)), np.zeros((m, top))
    for t in range(m):
        out = np.isnan(l[t]) | np.isneginf(l[t])
        rank = np.lexsort((np.arange(e), -np.where(out, -np.inf, l[t] + 0.0), out))
        chosen = [c for c in rank[:top] if not out[c]]
        ids[t, :len(chosen)] = chosen
        if not chosen:
            continue
        if np.isnan(l[t]).any() or np.isposinf(l[t]).any():
            weights[t, :len(chosen)] = np.nan
            continue
        d = np.where(out, -np.inf, l[t]) - l[t][chosen[0]]
        all_e = np.exp(d)
        part = np.array(chosen) if renorm else np.arange(e)
        z = all_e[part].sum()
        finite = np.where(np.isneginf(d), 0.0, np.abs(d))
        z_steps = (all_e[part] * (finite[part] + 6)).sum() / z + 22
        weights[t, :len(chosen)] = all_e[chosen] / z
        steps[t, :len(chosen)] = finite[chosen] + 6 + z_steps + 2
    return ids, weights, steps


def group_rows(ids, groups):
    """(offsets, order): rows sorted by group, the others last."""
    g = np.where((ids < 0) | (ids >= groups), groups, ids)
    order = np.argsort(g, kind="stable")
    return np.concatenate([[0], np.cumsum(np.bincount(g, minlength=groups + 1)[:groups])]), order


def half_step(v, eps, tiny):
    """Half a step of a type with relative spacing eps around v; no finer than half of `tiny`."""
    return np.maximum(np.abs(v) * eps / 2, tiny / 2)


def expert_products(w, ws, x, ids, top):
    """(p [slots, n], T = sum |terms|) of 64-bit x [rows, k] and experts' MXFP4 weights; zeros for slots of no group."""
    slots, n = len(ids), w.shape[1]
    p, total = np.zeros((slots, n)), np.zeros((slots, n))
    for e in np.unique(ids):
        if 0 <= e < w.shape[0]:
            at = np.nonzero(ids == e)[0]
            v = layer_ref.mxfp4_values(w[e], ws[e])
            p[at], total[at] = x[at // top] @ v.T, np.abs(x[at // top]) @ np.abs(v).T
    return p, total


def gated(p, err):
    """(silu(gate) * up, its error) of products with errors `err`; none of a slot without a group.

    silu's slope is below 1.1.  Its own evaluation: the exponential (six steps of 2^-24), the addition, the division
    and the product with the other half.
    """
    n = p.shape[1] // 2
    g, u = p[:, :n], p[:, n:]
    with np.errstate(over="ignore"):
        s = g / (1 + np.exp(-g))
    eg, eu = err[:, :n], err[:, n:]
    y = s * u
    return y, 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 9 * 2.0 ** -24 * (np.abs(s) + 1.1 * eg) * (np.abs(u) + eu)
