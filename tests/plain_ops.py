"""Plain 64-bit forms of the append and verification operators, in numpy, for
the tests (the attention's is the oracle's)."""
import numpy as np
import torch

import oracle

# half a step of a rounding to each storage type, relative to the value
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "f32": 2.0 ** -149}   # half of the least step


def normed(x, w, eps):
    """x [T, h, D] in 64 bits, normalised per head where there is a weight."""
    x = np.asarray(x, dtype=np.float64)
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)


def rotated(x, table, positions, interleaved):
    """(x rotated, the size of each element's pair) in 64 bits."""
    R = 0 if table is None else table.shape[1]
    y, size = x.copy(), np.abs(x)
    if R == 0:
        return y, size
    row = np.asarray(table, dtype=np.float64)[np.asarray(positions)][:, None, :]
    c, s = row[..., : R // 2], row[..., R // 2:]
    ia = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
    ib = ia + 1 if interleaved else ia + R // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size


def stored_error_bound(y, size, dtype):
    """How far a stored result may be from y.  The rounding is off by HALF |y|.
    Before it, in fp32 (u = 2^-24): the norm's sum of squares has at most 20
    roundings in a row (16 elements of a lane and 4 exchanges), the mean and eps
    2 more, halved by the root, which is off by 4 u itself: 15 u.  Weight times
    cos or sin, that times the element, the sum of a pair's two and the norm's
    product: 4 u of the pair's size.  32 u of it covers both, the reciprocal of
    head_dim, and the rounding of a value that is off by that much."""
    return HALF[dtype] * np.abs(y) + 32 * 2.0 ** -24 * size + TINY[dtype]


_E4M3 = None


def e4m3_values(codes):
    """Values of E4M3 codes (uint8), the oracle's decoding as a table."""
    global _E4M3
    if _E4M3 is None:
        _E4M3 = oracle.e4m3_decode(np.arange(256, dtype=np.uint8))
    return _E4M3[np.asarray(codes)]


def e4m3_codes(x):
    """E4M3 codes of finite values: nearest, ties to even, saturating at 448."""
    x = np.clip(np.asarray(x, dtype=np.float32), -448, 448)
    return torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def e4m3_between(codes, z, slack):
    """Whether each code is the rounding of some value within slack of z."""
    lo, hi = (e4m3_values(e4m3_codes(x)) for x in (z - slack, z + slack))
    v = e4m3_values(codes)
    return (lo <= v) & (v <= hi)


def weight(p, q):
    """max(p - q, 0) rounded to binary32; negative, NaN and infinite count as 0."""
    with np.errstate(invalid="ignore", over="ignore"):
        d = np.float32(p) - np.fmax(np.float32(q), np.float32(0))
        w = np.fmax(d.astype(np.float32), np.float32(0))
    return np.where(w < np.inf, w, np.float32(0))


def verify(target, draft, tokens, accept_u, sample_u, query_start, width):
    """(out_tokens, num_accepted); target and draft float32 [rows, V]."""
    B, V = len(query_start) - 1, target.shape[1]
    out = np.full((B, width), -1, dtype=np.int32)
    acc = np.zeros(B, dtype=np.int32)
    for s in range(B):
        q0, q1 = int(query_start[s]), int(query_start[s + 1])
        if q0 < 0 or q1 <= q0 or q1 > len(tokens) or q1 - q0 > width:
            continue
        a, rejected = 0, False
        for r in range(q0 + 1, q1):
            x = int(tokens[r])
            ok = False
            if 0 <= x < V:
                p = weight(target[r - 1, x], 0.0)
                q = 1.0 if draft is None else np.fmax(draft[r, x], np.float32(0))
                ok = np.float64(accept_u[r]) * np.float64(q) < np.float64(p)
            if not ok:
                rejected = True
                break
            a += 1
        row = q0 + a
        p = target[row].astype(np.float32)
        w = weight(p, np.zeros_like(p))
        if rejected:
            left = w.copy()
            if draft is not None:
                left = weight(p, draft[row + 1].astype(np.float32))
            elif 0 <= tokens[row + 1] < V:
                left[tokens[row + 1]] = 0
            w = left if left.max() > 0 else w
        acc[s] = a
        out[s, :a] = tokens[q0 + 1: q0 + 1 + a]
        if w.max() > 0:
            c = np.cumsum(w.astype(np.float64))
            u = min(max(float(sample_u[s]), 0.0), 1.0) if sample_u[s] == sample_u[s] else 0.0
            v = int(np.searchsorted(c, u * c[-1], side="right"))
            out[s, a] = min(v, int(np.flatnonzero(w > 0)[-1]))
    return out, acc
