"""Plain 64-bit reference of the recent window (tests only): rotary positions, the window cache and
windowed attention, written from their definitions on numpy arrays."""
import decimal
import functools

import numpy as np

PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899863")

D, GROUP = 128, 32
Q = {8: 127, 4: 7}
STEP_TOP = {8: 56.0, 4: 896.0}


def bf16(x):
    """float64 -> the nearest bf16 values (ties to even), as float64."""
    f = np.asarray(x, np.float64)
    m, e = np.frexp(f)
    scale = np.ldexp(1.0, np.maximum(e, -125) - 8)
    return np.where(np.isfinite(f), np.rint(f / scale) * scale, f)


def rope(x, dims, theta, pairing, shared, positions, sign=1.0):
    """x [n][128] float64; positions int [n][3]."""
    out = np.array(x, np.float64)
    R, i = sum(dims), 0
    for a in range(3):
        for j in range(dims[a] // 2):
            rate = float(theta[a]) ** (-(2.0 * i / R if shared else 2.0 * j / dims[a]))
            ang = sign * np.remainder(positions[:, a].astype(np.longdouble) * np.longdouble(rate), 2 * np.pi).astype(np.float64)
            c0, c1 = (2 * i, 2 * i + 1) if pairing == "interleaved" else (i, i + R // 2)
            p, q = x[:, c0], x[:, c1]
            out[:, c0], out[:, c1] = p * np.cos(ang) - q * np.sin(ang), p * np.sin(ang) + q * np.cos(ang)
            i += 1
    return out


@functools.lru_cache(maxsize=None)
def exact_turns(dims, theta, shared, bits=200):
    """Every pair's part of a turn per unit of position, from 80 digits, as an integer over 2^bits."""
    out, i = [], 0
    with decimal.localcontext() as c:
        c.prec = 80
        for a in range(3):
            for j in range(dims[a] // 2):
                e = decimal.Decimal(2 * i) / sum(dims) if shared else decimal.Decimal(2 * j) / dims[a]
                out.append(int(decimal.Decimal(theta[a]) ** -e / (2 * PI) * 2 ** bits))
                i += 1
    return out


def grid_positions(start, n, gh, gw):
    p = np.arange(start, start + n, dtype=np.int64)
    return np.stack([p // (gh * gw), p // gw % gh, p % gw], 1)


def steps(bits):
    """Every step by its byte."""
    s = (np.arange(248, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    return s[s <= STEP_TOP[bits]]


def quantise(x, bits):
    """x [n][128] float64 (finite, in range) -> signed codes int [n][128], step bytes [n][4]."""
    table = steps(bits)
    g = np.asarray(x, np.float64).reshape(-1, D // GROUP, GROUP)
    step = np.minimum(np.searchsorted(table * Q[bits], np.abs(g).max(-1)), len(table) - 1)
    s = table[step][..., None]
    q = np.where(s > 0, np.rint(g / np.where(s > 0, s, 1.0)), 0.0)
    return np.clip(q, -Q[bits], Q[bits]).reshape(-1, D).astype(np.int64), step.astype(np.uint8)


def pack(q, bits):
    if bits == 8:
        return (q + 128).astype(np.uint8)
    out = np.zeros((q.shape[0], D // 2), np.uint8)
    for c in range(D):
        j, k, t = c // 8, c % 8 // 2, c % 2
        nib = k + 4 * t
        out[:, 4 * j + nib // 2] |= ((q[:, c] + 8).astype(np.uint8) << (4 * (nib % 2))).astype(np.uint8)
    return out


def values(codes, step, bits):
    """Packed rows [n][..], step bytes [n][4] -> float64 [n][128]."""
    c = np.asarray(codes).astype(np.int64)
    if bits == 8:
        q = c - 128
    else:
        q = np.zeros((c.shape[0], D), np.int64)
        for ch in range(D):
            j, k, t = ch // 8, ch % 8 // 2, ch % 2
            nib = k + 4 * t
            q[:, ch] = ((c[:, 4 * j + nib // 2] >> (4 * (nib % 2))) & 15) - 8
    s = (np.asarray(step).astype(np.uint16) << 7).view(np.float16).astype(np.float64)
    return q * np.repeat(s, GROUP, 1)


def slot_of(p, sink, ring):
    return p if p < sink else sink + (p - sink) % ring


def held(length, sink, ring):
    return [p for p in range(length) if p < sink or p >= length - ring]


def attend(q, k, v, pos, q_start, tpf, frames, sink, scale):
    """One head: q [nq][d] at positions q_start + i, keys k, v [m][d] at positions pos [m] (float64).
    Returns out [nq][d], lse [nq] (log2), and per row the error scales: max over keys of
    sum_c |q_c k_c| scale log2(e), and sum_j w_j |v_j| [nq][d]."""
    nq, m = len(q), len(k)
    out, lse = np.zeros((nq, D)), np.full(nq, -np.inf)
    mag, spread = np.zeros(nq), np.zeros((nq, D))
    if m == 0:
        return out, lse, mag, spread
    fk = pos // tpf
    for i in range(nq):
        f = (q_start + i) // tpf
        see = (fk <= f) & ((f - fk < frames) | (pos < sink))
        if not see.any():
            continue
        x = (k[see] @ q[i]) * scale * np.log2(np.e)
        mx = x.max()
        w = np.exp2(x - mx)
        lse[i] = mx + np.log2(w.sum())
        w /= w.sum()
        out[i], spread[i] = w @ v[see], w @ np.abs(v[see])
        mag[i] = (np.abs(k[see]) @ np.abs(q[i])).max() * scale * np.log2(np.e)
    return out, lse, mag, spread
