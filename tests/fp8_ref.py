"""Plain references for the fp8 (e4m3) layer and the token read-out: numpy,
64 bits, written from the formats' and operators' definitions.  Used by the
tests only."""
import numpy as np


def e4m3_values():
    """The 256 values of OCP e4m3 in code order, as float64 (NaN at 0x7f and 0xff)."""
    v = np.empty(256)
    for code in range(256):
        sign, exp, man = code >> 7, (code >> 3) & 15, code & 7
        x = np.ldexp(1 + man / 8, exp - 7) if exp else np.ldexp(man / 8, -6)
        if code & 127 == 127:
            x = np.nan
        v[code] = -x if sign else x
    return v


E4M3 = e4m3_values()
_POS = E4M3[:127]                       # 0 ... 448, ascending
_MID = (_POS[1:] + _POS[:-1]) / 2       # rounding ties, exact in float64


def round_e4m3(x):
    """float -> the nearest e4m3 value (ties to the even code), clamped to +-448; float64 array."""
    a = np.minimum(np.abs(np.asarray(x, np.float64)), 448.0)
    lo = np.searchsorted(_MID, a, side="left")       # a <= _MID[lo]: below or at the tie above code lo
    at_tie = (lo < len(_MID)) & (a == _MID[np.minimum(lo, len(_MID) - 1)])
    code = lo + (at_tie & (lo % 2 == 1))
    return np.copysign(_POS[code], x)


def _grouped(x, rows):
    """x [m, k] -> zero-padded groups [m/rows, rows, KB, 128]."""
    m, k = x.shape
    p = np.zeros((-(-m // rows) * rows, -(-k // 128) * 128), x.dtype)
    p[:m, :k] = x
    return p.reshape(p.shape[0] // rows, rows, p.shape[1] // 128, 128)


def quantize(x, rows):
    """fp32 x [m, k] -> (values of the codes float64 [m, k], scales fp32 [groups, KB]); the definition step by step,
    x / s in fp32 (IEEE division)."""
    x = np.asarray(x, np.float32)
    m, k = x.shape
    g = _grouped(x, rows)
    with np.errstate(all="ignore"):
        a = np.abs(g).max(axis=(1, 3))
        bad = ~np.isfinite(g).all(axis=(1, 3))
        s = (a / np.float32(448)).astype(np.float32)
        s[bad] = np.nan
        sb = s[:, None, :, None]
        t = (g / sb).astype(np.float32)
        t = np.where(sb > 0, t, np.float32(0))
    v = round_e4m3(t)
    return v.reshape(-1, v.shape[2] * 128)[:m, :k], s


def swiglu(gate, up):
    g = np.asarray(gate, np.float64)
    with np.errstate(all="ignore"):
        return g / (1 + np.exp(-g)) * np.asarray(up, np.float64)


def spread(s, k, rows=None, m=None):
    """Scales over their values: [KB, M] -> [M, k] (rows None), or tile scales [NB, KB] -> [m, k]."""
    col = np.arange(k) // 128
    if rows is None:
        return np.asarray(s, np.float64).T[:, col]
    return np.asarray(s, np.float64)[np.arange(m) // rows][:, col]


def gemm(q, s_a, w, s_w):
    """Code values q [M, K], w [N, K]; s_a [KB, M], s_w [NB, KB] -> (y, sum of magnitudes, per-block largest
    products summed) in float64."""
    a = np.asarray(q, np.float64) * spread(s_a, q.shape[1])
    b = np.asarray(w, np.float64) * spread(s_w, w.shape[1], 128, w.shape[0])
    return a @ b.T, np.abs(a) @ np.abs(b).T


def block_peaks(q, s_a, w, s_w):
    """sum over blocks of (largest |q| of the row's block) (largest |w| of the column's block) s_a s_w: at least the
    sum over blocks of the largest product."""
    a = np.abs(np.asarray(q, np.float64) * spread(s_a, q.shape[1]))
    b = np.abs(np.asarray(w, np.float64) * spread(s_w, w.shape[1], 128, w.shape[0]))
    pa = _grouped(a, 1).max(axis=(1, 3))
    pb = _grouped(b, 1).max(axis=(1, 3))
    return pa @ pb.T


def logprobs(z, tokens, top):
    """(logprobs, lse, entropy, top ids, top logprobs) of fp32 logits [M, V], in float64."""
    z = np.asarray(z, np.float64)
    M, V = z.shape
    T = tokens.shape[1]
    lp = np.full((M, T), np.nan)
    lse, ent = np.full(M, np.nan), np.full(M, np.nan)
    ids, tlp = np.full((M, top), -1, np.int64), np.full((M, top), np.nan)
    for r in range(M):
        row = z[r]
        if np.isnan(row).any() or (row == np.inf).any():
            continue
        m = row.max()
        if m == -np.inf:
            lse[r], ent[r] = -np.inf, 0.0
            full = row
        else:
            e = np.exp(row - m)
            lse[r] = m + np.log(e.sum())
            full = (row - m) - np.log(e.sum())
            live = e > 0
            ent[r] = -(np.exp(full[live]) * full[live]).sum()
        for i in range(T):
            if 0 <= tokens[r, i] < V:
                lp[r, i] = full[tokens[r, i]]
        order = np.argsort(-row, kind="stable")[:top]
        order = order[full[order] > -np.inf]
        ids[r, :len(order)] = order
        tlp[r] = -np.inf
        tlp[r, :len(order)] = full[order]
    return lp, lse, ent, ids, tlp
