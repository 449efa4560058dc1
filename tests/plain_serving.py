"""Plain 64-bit forms of the 4-bit cache, of building a step and of processed
logits, in numpy, for the tests."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """Values of the 256 E4M3 codes, from the format's definition."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(c >> 7, -v, v)


def nearest(x, values):
    """Index of the nearest of ascending values (of x >= 0), ties to the even index,
    saturating."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    down, up = x - values[lo], values[hi] - x
    take_up = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.where(take_up, hi, lo)


def fp4_quantise(x, scale):
    """(codes [.., D], scale codes [.., D/16]) of float32 x [T, h, D], scale [h]."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        y = (np.asarray(x, np.float32) / np.asarray(scale, np.float32)[:, None]).astype(np.float32)
        y = y.reshape(*y.shape[:-1], -1, 16)
        nan = np.isnan(y).any(-1)
        top = np.abs(np.where(np.isnan(y), 0, y)).max(-1)
        q = (top / np.float32(6)).astype(np.float32)
    e4m3 = e4m3_values()[:127]                     # 0 .. 448
    sc = nearest(np.minimum(q, np.float32(448)), e4m3)
    S = e4m3[sc].astype(np.float32)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        z = np.where(S[..., None] > 0, y / S[..., None], np.float32(0)).astype(np.float32)
    z = np.where(np.isnan(z), 0, z)
    codes = nearest(np.minimum(np.abs(z), 6), E2M1) + 8 * np.signbit(z)
    codes = np.where(nan[..., None], 0, codes)
    sc = np.where(nan, 127, sc)
    return codes.reshape(*codes.shape[:-2], -1).astype(np.uint8), sc.astype(np.uint8)


def fp4_values(codes, sc, scale):
    """Values in 64 bits: codes [.., h, D] (0..15), sc [.., h, D/16], scale [h]."""
    v = np.where(codes >> 3, -1.0, 1.0) * E2M1[codes & 7]
    v = v.reshape(*v.shape[:-1], -1, 16) * e4m3_values()[sc][..., None]
    return v.reshape(codes.shape) * np.asarray(scale, np.float64)[:, None]


def fp4_unpack(cache):
    """(codes [N, h, 16, D], scale codes [N, h, 16, D/16]) of uint8 tiles [N, h, 9, D]."""
    N, h, _, D = cache.shape
    b = cache[:, :, :8].reshape(N, h, 16, D // 2)
    codes = np.stack([b & 15, b >> 4], -1).reshape(N, h, 16, D)
    return codes, cache[:, :, 8].reshape(N, h, 16, D // 16)


def fp4_write(cache, x, scale, slots):
    """cache with the rows x [T, h, D] written at their slots."""
    out = cache.copy()
    N, h, _, D = cache.shape
    codes, sc = fp4_quantise(x, scale)
    c, s = out[:, :, :8].reshape(N, h, 16, D // 2), out[:, :, 8].reshape(N, h, 16, D // 16)
    for t, slot in enumerate(slots):
        if 0 <= slot < N * 16:
            c[slot // 16, :, slot % 16] = codes[t, :, ::2] | (codes[t, :, 1::2] << 4)
            s[slot // 16, :, slot % 16] = sc[t]
    out[:, :, :8] = c.reshape(N, h, 8, D)
    out[:, :, 8] = s.reshape(N, h, D)
    return out


def fp4_cache_values(cache, scale):
    """[N, h, 16, D] in 64 bits."""
    codes, sc = fp4_unpack(cache)
    return fp4_values(codes.transpose(0, 2, 1, 3), sc.transpose(0, 2, 1, 3), scale).transpose(0, 2, 1, 3)


def blocks_for(n):
    return -(-int(n) // 16)


def named_twice(ids, R):
    ids = [] if ids is None else [int(i) for i in ids if 0 <= i < R]
    return len(set(ids)) < len(ids)


def build_step(st, ids, ctx, new, width, num_rows, num_blocks):
    """One step, sequence by sequence; st: dict of request_tables, request_blocks,
    free_blocks, free_count (numpy, changed in place; free_blocks None: no list).
    Returns the outputs (table entries that are not written: None)."""
    B = len(ctx)
    R, RW = st["request_tables"].shape
    count = int(st["free_count"][0]) if st["free_blocks"] is not None else 0
    tables = np.full((B, width), -7, dtype=np.int64)         # -7: not written
    lens = np.zeros(B, np.int64)
    starts = np.zeros(B + 1, np.int64)
    pos, slots = np.zeros(num_rows, np.int64), np.full(num_rows, -1, np.int64)
    total, asked, taken, flags = 0, 0, 0, 0
    old_tables, old_blocks = st["request_tables"].copy(), st["request_blocks"].copy()
    twice = named_twice(ids, R)
    if twice:
        flags |= 0x2
    for s in range(B):
        i = s if ids is None else int(ids[s])
        c, n = int(ctx[s]), 1 if new is None else int(new[s])
        starts[s] = min(total, num_rows)
        rows = max(n, 0)
        ok = 0 <= i < R and c >= 0 and n >= 0 and c + n <= 16 * min(width, RW)
        ok = ok and 0 <= old_blocks[i] <= RW
        need = 0
        if ok:
            need = max(blocks_for(c + n) - int(old_blocks[i]), 0)
            asked += need
        if not ok or total + rows > num_rows:
            ok = False
            if ids is None or i != -1 or total + rows > num_rows:
                flags |= 0x2
        elif need and asked > count:
            ok = False
            flags |= 0x40
        table = None
        ok = ok and not twice
        if ok:
            table = [int(x) for x in old_tables[i]]
            for k in range(need):
                b = int(st["free_blocks"][count - 1 - (asked - need + k)])
                e = int(old_blocks[i]) + k
                table[e] = b
                st["request_tables"][i, e] = b
            if need:
                taken = asked
                st["request_blocks"][i] = old_blocks[i] + need
            w = blocks_for(c + n)
            tables[s, :w] = table[:w]
            lens[s] = c + n
        for k in range(rows):
            r = total + k
            if r >= num_rows:
                break
            p = c + k
            pos[r] = p
            if ok:
                b = table[p // 16]
                if 0 <= b < num_blocks:
                    slots[r] = b * 16 + p % 16
                else:
                    flags |= 0x1
        total += rows
    starts[B] = min(total, num_rows)
    if taken:
        st["free_count"][0] = count - taken
    return dict(tables=tables, lens=lens, starts=starts, positions=pos, slots=slots, flags=flags)


def trim(st, ids, keep):
    """Blocks past keep given back, in place; returns the error flags."""
    R, RW = st["request_tables"].shape
    flags, back = 0, []
    twice = named_twice(ids, R)
    for s in range(len(keep)):
        i = s if ids is None else int(ids[s])
        if ids is not None and i == -1:
            continue
        if not 0 <= i < R or keep[s] < 0 or not 0 <= st["request_blocks"][i] <= RW:
            flags |= 0x2
            continue
        k = min(int(st["request_blocks"][i]), blocks_for(keep[s]))
        back.append((i, k, [int(x) for x in st["request_tables"][i, k:st["request_blocks"][i]]]))
    if twice:
        return flags | 0x2
    given = [b for _, _, bs in back for b in bs]
    count = int(st["free_count"][0])
    if count + len(given) > len(st["free_blocks"]):
        return flags | 0x1
    st["free_blocks"][count:count + len(given)] = given[::-1]
    st["free_count"][0] = count + len(given)
    for i, k, bs in back:
        if bs:
            st["request_blocks"][i] = k
    return flags


def logits(x, starts, tokens=None, history=None, prompt_lens=None, history_lens=None,
           repetition=None, frequency=None, presence=None, bias=None, allowed=None,
           temperature=None, probs=True):
    """Rows of sequences in 64 bits (rows of none: NaN); bias: per sequence a list of
    (token, value); allowed: bool [T, V]."""
    T, V = x.shape
    out = np.full((T, V), np.nan)
    for s in range(len(starts) - 1):
        for r in range(starts[s], starts[s + 1]):
            z = x[r].astype(np.float64)
            prompt, said = [], []
            if history is not None:
                p = 0 if prompt_lens is None else prompt_lens[s]
                prompt, said = list(history[s][:p]), list(history[s][p:history_lens[s]])
            if tokens is not None:
                said += list(tokens[starts[s] + 1:r + 1])
            n = np.bincount([v for v in said if 0 <= v < V], minlength=V)
            seen = (n + np.bincount([v for v in prompt if 0 <= v < V], minlength=V)) > 0
            th = 1.0 if repetition is None else float(repetition[s])
            al = 0.0 if frequency is None else float(frequency[s])
            be = 0.0 if presence is None else float(presence[s])
            if th != 1 or al != 0 or be != 0:
                z = np.where(seen, np.where(z > 0, z / th, z * th), z)
                z = z - al * n - be * (n > 0)
            if bias is not None:
                for v, b in bias[s]:
                    if 0 <= v < V:
                        z[v] += float(b)
            if allowed is not None:
                z = np.where(allowed[r], z, -np.inf)
            tau = 1.0 if temperature is None else float(temperature[s])
            if tau > 0:
                z = z / tau
            if probs:
                top = np.max(z[~np.isnan(z)], initial=-np.inf)
                if not tau > 0:
                    e = np.zeros(V)
                    if top > -np.inf:
                        e[np.flatnonzero(z == top)[0]] = 1
                    z = e
                else:
                    with np.errstate(invalid="ignore"):
                        e = np.exp(z - (top if top > -np.inf else 0.0))
                        z = e / e.sum() if e.sum() != 0 else np.zeros(V)
            out[r] = z
    return out
