"""Plain references for the mixture-of-experts operators: numpy, 64 bits, from their definitions.  Used by the tests
only."""
import numpy as np

import fp8_ref


def norm(h, gain, eps):
    """h fp32 [M, K] (already added and rounded) -> y fp32: inv in 64 bits rounded once, two fp32 products."""
    h = np.asarray(h, np.float32)
    with np.errstate(all="ignore"):
        s = np.square(h.astype(np.float64)).sum(1) / h.shape[1]
        inv = (1 / np.sqrt(s + eps)).astype(np.float32)
        return (h * inv[:, None]).astype(np.float32) * np.asarray(gain, np.float32)


def quantize_int8(y):
    """fp32 [M, K] -> (codes int8, scales fp32 [M])."""
    y = np.asarray(y, np.float32)
    with np.errstate(all="ignore"):
        s = np.abs(y).max(1) * (np.float32(1) / np.float32(127))
        s[~np.isfinite(y).all(1)] = np.nan
        t = np.where(s[:, None] > 0, (y / s[:, None]).astype(np.float32), np.float32(0))
        return np.clip(np.rint(t), -127, 127).astype(np.int8), s


def quantize_fp8(y):
    """fp32 [M, K] -> (values of the codes, scales [KB, M])."""
    v, s = fp8_ref.quantize(y, 1)
    return v, np.ascontiguousarray(s.T)


def route(z, top, score="softmax", bias=None, renormalize=True, scale=1.0):
    """(ids, weights in 64 bits, offsets, rows, slots) of logits [M, E], token by token."""
    z = np.asarray(z, np.float64)
    M, E = z.shape
    ids, weights = np.full((M, top), -1, np.int64), np.zeros((M, top))
    for m in range(M):
        row = z[m]
        if np.isnan(row).any() or (row == np.inf).any():
            weights[m] = np.nan
            continue
        most = row.max()
        if most == -np.inf:
            continue
        with np.errstate(over="ignore"):
            if score == "softmax":
                e = np.exp(row - most)
                s = e / e.sum()
            else:
                s = 1 / (1 + np.exp(-row))
        key = row.copy()
        if bias is not None:
            key = np.where(row > -np.inf, s + np.asarray(bias, np.float64), -np.inf)
            key[np.isnan(key)] = -np.inf
        order = np.argsort(-key, kind="stable")[:top]
        order = order[key[order] > -np.inf]
        w = s[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        ids[m, :len(order)] = order
        weights[m, :len(order)] = w * np.float64(np.float32(scale))
    return (ids, weights) + dispatch(ids, E)


def dispatch(ids, E):
    """(offsets, rows, slots): the list of all choices by expert, then by token."""
    M, top = ids.shape
    rows, slots, offsets = np.full(M * top, -1, np.int64), np.full((M, top), -1, np.int64), [0]
    at = 0
    for e in range(E):
        for m, j in np.argwhere(ids == e):
            rows[at] = m
            slots[m, j] = at
            at += 1
        offsets.append(at)
    return np.array(offsets), rows, slots


def combine(x, weights, slots, add=None):
    """(y, sum of magnitudes) in 64 bits."""
    x, weights = np.asarray(x, np.float64), np.asarray(weights, np.float64)
    M, top = slots.shape
    y = np.zeros((M, x.shape[1])) if add is None else np.asarray(add, np.float64).copy()
    mag = np.abs(y)
    for j in range(top):
        live = (slots[:, j] >= 0) & (slots[:, j] < len(x))
        part = np.zeros_like(y)
        part[live] = x[slots[live, j]]
        with np.errstate(invalid="ignore"):
            y += weights[:, j, None] * part
            mag += np.abs(weights[:, j, None] * part)
    return y, mag
