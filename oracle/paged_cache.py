"""The 4-bit paged cache in fp64 numpy: number formats by their definition,
byte positions, lengths-to-tables bookkeeping and attention.  Test
infrastructure; shares no code with the kernels."""
import math

import numpy as np

#: E2M1 (two exponent bits, one fraction bit, bias 1), by code 0..7; bit 3 is the sign.
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3(byte):
    """Value of a non-negative E4M3 byte (bias 7; 0x7f is NaN)."""
    byte = np.asarray(byte, dtype=np.int64)
    e, m = byte >> 3 & 15, byte & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    return np.where(byte == 0x7f, np.nan, v)


E4M3 = e4m3(np.arange(0x7f))  # 0 .. 448


def nearest(grid, x):
    """Index of the nearest grid value, ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    up, down = grid[hi] - x, x - grid[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x):
    """x [..., 16 n] fp64 -> (codes [..., 16 n], scale bytes [..., n])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    mag = np.abs(b)
    sb = nearest(E4M3, mag.max(-1) / 6)
    s = E4M3[sb][..., None]
    idx = np.zeros(b.shape, dtype=np.int64)
    mids = (E2M1[1:] + E2M1[:-1]) / 2
    for i, mid in enumerate(mids):
        idx += (mag > mid * s) | ((mag == mid * s) & (i % 2 == 1))
    idx = np.where(s > 0, idx, 0)
    return (idx | np.where((b < 0) & (s > 0), 8, 0)).reshape(x.shape), sb


def dequantise(codes, scales):
    """The inverse of ``quantise``."""
    c = codes.reshape(*scales.shape, 16)
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0) * e4m3(scales)[..., None]
    return v.reshape(codes.shape)


def offsets(D, i, c):
    """Byte offsets in a group of 16 tokens: K code, V code, K scale, V scale of
    token i, channel c."""
    b, n = c // 16, D // 64
    return (i * D // 2 + c // 2,
            8 * D + i // 8 * 4 * D + b * 64 + i % 8 * 8 + c % 16 // 2,
            16 * D + i % 8 * (D // 8) + b // n * 2 * n + i // 8 * n + b % n,
            17 * D + 16 * b + i % 8 // 2 * 4 + i // 8 * 2 + i % 2)


def _index(D):
    i, c = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
    return offsets(D, i, c)


def store(cache, slots, k, v):
    """Write k, v [T, heads, D] (fp64) at slots into cache [pages, heads, P / 16, 18 D]."""
    T, H, D = k.shape
    P = cache.shape[2] * 16
    slots = np.asarray(slots, dtype=np.int64)
    page, tok = slots // P, slots % P
    flat = cache.reshape(-1)
    assert flat.base is not None  # a view: the writes land in the cache
    base = ((page[:, None] * H + np.arange(H)) * (P // 16) + tok[:, None] // 16) * 18 * D
    kc, vc, ks, vs = _index(D)
    i = tok % 16
    for x, code_at, scale_at in ((k, kc, ks), (v, vc, vs)):
        codes, sb = quantise(x)
        flat[base[..., None] + code_at[i, None, ::2]] = codes[..., 0::2] | codes[..., 1::2] << 4
        flat[base[..., None] + scale_at[i, None, ::16]] = sb


def load_group(group):
    """K, V [16, D] fp64 of one group's 18 D bytes."""
    D = group.shape[-1] // 18
    kc, vc, ks, vs = _index(D)
    shift = np.arange(D) % 2 * 4
    out = []
    for code_at, scale_at in ((kc, ks), (vc, vs)):
        c = group[code_at].astype(np.int64) >> shift & 15
        out.append(E2M1[c & 7] * np.where(c & 8, -1.0, 1.0) * e4m3(group[scale_at] & 0x7f))
    return out


def tables(held, seq, new, table, ring, span, P, max_tokens):
    """The contract of kda_cache_tables in a loop.  Returns (kv, cu, slots, span,
    table, ring, error)."""
    held, seq, new = (list(map(int, x)) for x in (held, seq, new))
    table, ring = np.array(table), np.array(ring)
    head, tail = map(int, span)
    err = False
    if head < 0 or tail < head or tail - head > len(ring):
        head = tail = 0
        err = True
    avail = tail - head
    kv, cu, slots, asked, blocks = [], [0], [], 0, table.shape[1]
    start, end = head, tail
    for b in range(len(held)):
        add = max(new[b], 0)
        cu.append(cu[-1] + add)
        have = -(-held[b] // P)
        if held[b] < 0 or seq[b] < 0 or seq[b] > held[b] or new[b] < -1 or have > blocks:
            kv.append(0)
            slots += [-1] * add
            err = True
            continue
        keep = seq[b] if new[b] >= 0 else 0
        want = -(-(keep + add) // P)
        ok = want <= blocks
        if ok:
            asked += max(0, want - have)
            ok = want <= have or asked <= avail
        if not ok:
            err, want = True, -(-keep // P)
        for j in range(want, have):
            ring[end % len(ring)] = table[b, j]
            end += 1
        for j in range(have, want):
            table[b, j] = ring[start % len(ring)]
            start += 1
        kv.append(keep + add if ok else keep)
        slots += [int(table[b, p // P]) * P + p % P for p in range(keep, keep + add)] if ok \
            else [-1] * add
    err = err or len(slots) > max_tokens or end - start > len(ring)
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    return kv, cu, slots, (start, end), table, ring, err


def attention(q, ks, vs, scale):
    """One request: q [n, Hq, D], ks, vs [L, Hk, D] fp64 (the n new tokens last).
    Returns out [n, Hq, D], lse [n, Hq], and for error bounds sum p|v| [n, Hq, D],
    sum |v| / sum exp(s - max) [n, Hq, D] and max_j scale sum_c |q_c k_jc| [n, Hq]."""
    n, Hq, D = q.shape
    L, Hk = ks.shape[:2]
    out, mass = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    flat, size = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    lse = np.full((n, Hq), -math.inf)
    for i in range(n):
        see = L - n + i + 1
        if see <= 0:
            continue
        for h in range(Hq):
            k, v = ks[:see, h * Hk // Hq], vs[:see, h * Hk // Hq]
            s = k @ q[i, h] * scale
            top = s.max()
            p = np.exp(s - top)
            z = p.sum()
            out[i, h] = p @ v / z
            mass[i, h] = p @ np.abs(v) / z
            flat[i, h] = np.abs(v).sum(0) / z
            size[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * abs(scale)
            lse[i, h] = top + math.log(z)
    return out, lse, mass, flat, size
