"""Plain numpy models, in 64 bits, of the calls on rows grouped by adapter or expert."""
import numpy as np


def plan(ids, E):
    """(offs, order, pos, units) of ids [T, top_k] or [T], as mmq.h defines the plan's regions."""
    flat = np.asarray(ids).reshape(-1)
    P = flat.size
    key = np.where((flat >= 0) & (flat < E), flat, E).astype(np.int64)
    order = np.argsort(key, kind="stable")
    count = np.bincount(key, minlength=E + 1)
    offs = np.concatenate([[0], np.cumsum(count)])
    pos = np.full(P, -1, np.int64)
    n = int(offs[E])
    pos[order[:n]] = np.arange(n)
    units = []
    for g in range(E + 1):
        for first in range(int(offs[g]), int(offs[g + 1]), 64):
            units.append((g, first, min(64, int(offs[g + 1]) - first), 0))
    full = np.zeros((P // 64 + min(E + 1, P), 4), np.int64)
    if units:
        full[:len(units)] = units
    return offs[:E + 1], order, pos, full


def row_of(ids, E, order):
    """The row of each pair ([T, top_k]) in a row buffer of `order`, -1 for a pair without one."""
    ids = np.asarray(ids)
    pos = plan(ids, E)[2]
    row = pos if order == "sorted" else np.where(pos >= 0, np.arange(ids.size), -1)
    return row.reshape(ids.shape)


def bf16(x):
    """x rounded to bf16 (nearest even), as f32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


# ------------------------------------------------------------------------------ adapters

def act_values(kind, q, s):
    """x^ [M, K] in 64 bits from int8 values q [M, K] and the scales ([M, K/32], or [M])."""
    s = np.asarray(s, np.float64)
    per = np.repeat(s, 32, axis=1) if kind == "q8_1" else s[:, None]
    return q.astype(np.float64) * per


def lora(x, A, B, scale, ids, base):
    """(out, v) and the sums of the terms' magnitudes (out, v) behind them."""
    M, R = x.shape[0], A.shape[1]
    out, v = np.array(base, np.float64), np.zeros((M, R))
    mag_out, mag_v = np.abs(out), np.zeros((M, R))
    for e in range(A.shape[0]):
        at = np.nonzero(ids == e)[0]
        v[at] = x[at] @ A[e].T
        mag_v[at] = np.abs(x[at]) @ np.abs(A[e]).T
        out[at] += scale[e] * (v[at] @ B[e].T)
        mag_out[at] += abs(scale[e]) * (mag_v[at] @ np.abs(B[e]).T)
    return out, v, mag_out, mag_v


def lora_grad(x, A, B, scale, ids, v, dy, dx_base):
    """(dx, dA, dB) and the sums of the terms' magnitudes behind each."""
    res = [np.array(dx_base, np.float64), np.zeros(A.shape), np.zeros(B.shape)]
    mag = [np.abs(res[0]), np.zeros(A.shape), np.zeros(B.shape)]
    for e in range(A.shape[0]):
        at = np.nonzero(ids == e)[0]
        for to, f in ((res, lambda a: a), (mag, np.abs)):
            u = f(scale[e]) * (f(dy[at]) @ f(B[e]))
            to[0][at] += u @ f(A[e])
            to[1][e] = u.T @ f(x[at])
            to[2][e] = f(scale[e]) * (f(dy[at]).T @ f(v[at]))
    return res, mag


def full_significands(r, n, bits):
    """n values in [1, 2) of `bits` significand bits: random ones, and ones whose upper parts end in
    ones, 1 + 2^-7 - 2^(1 - bits)."""
    v = r.integers(1 << (bits - 1), 1 << bits, n)
    v[::3] = (1 << (bits - 1)) + (1 << (bits - 8)) - 1
    return v
