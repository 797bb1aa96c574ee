"""The 8-bit paged cache in fp64 numpy, and the bookkeeping of pages that several rows
hold, by their definitions.  Test infrastructure; shares no code with the kernels."""
import math

import numpy as np

from oracle.paged_cache import E4M3, e4m3, nearest

LEAST, MOST = -100, 119  # exponents: of a block of zeros; 448 2^MOST is the last that fp32 holds


def exponent(top):
    """The least e >= LEAST with top <= 448 2^e, MOST at most."""
    if top <= 448.0 * 2.0 ** LEAST:
        return LEAST
    e = math.ceil(math.log2(top / 448.0))
    while top > 448.0 * 2.0 ** e:
        e += 1
    while top <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return min(e, MOST)


def code(x, e):
    """E4M3 bytes of x / 2^e: nearest, ties to even, saturating; NaN gives 0."""
    x = np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=np.inf, neginf=-np.inf)
    b = nearest(E4M3, np.minimum(np.abs(x) * 2.0 ** -e, 448.0))
    return b | np.where(np.signbit(x), 128, 0)


def value(byte, e=0):
    """What codes stand for."""
    byte = np.asarray(byte).astype(np.int64)
    return np.where(byte & 128, -1.0, 1.0) * e4m3(byte & 127) * 2.0 ** e


def offsets(D, i, c):
    """Byte of K's and of V's code of token i, channel c, in a block's 32 D + 16 bytes."""
    k = c % (D // 4) // 16 * 1024 + i * 64 + c // (D // 4) * 16 + c % 16
    v = 16 * D + (i // 8 * 2 + i % 2) * 4 * D + c // (D // 8) * (D // 2) + \
        i % 8 // 2 * (D // 8) + c % (D // 8)
    return k, v


def index(D):
    i, c = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
    return offsets(D, i, c)


def store(cache, slots, k, v):
    """Append k, v [T, heads, D] (fp64) at slots to cache [pages, heads, P / 16, 32 D + 16]."""
    T, H, D = k.shape
    P = cache.shape[2] * 16
    slots = [int(s) for s in slots]
    t = 0
    while t < T:
        end = t + 1
        while end < T and slots[t] >= 0 and slots[end] // 16 == slots[t] // 16:
            end += 1
        if slots[t] >= 0:
            places = [s % 16 for s in slots[t:end]]
            for h in range(H):
                block = cache[slots[t] // P, h, slots[t] % P // 16]
                for n, x in enumerate((k, v)):
                    new = x[t:end, h]
                    mag = np.abs(new[np.isfinite(new)])
                    e = exponent(float(mag.max()) if mag.size else 0.0)
                    at = index(D)[n]
                    if 0 not in places:
                        old = int(block[32 * D + n]) - 127
                        if e > old:
                            for i in range(16):
                                if i not in places:
                                    held = value(block[at[i]], old)  # a code of NaN stays one
                                    block[at[i]] = np.where(np.isnan(held), block[at[i]],
                                                            code(held, e))
                        e = max(e, old)
                    for j, i in enumerate(places):
                        block[at[i]] = code(new[j], e)
                    block[32 * D + n] = e + 127
        t = end


def load_block(block):
    """K, V [16, D] fp64 of a block's bytes."""
    D = (block.shape[-1] - 16) // 32
    return [value(block[at], float(block[32 * D + n]) - 127) for n, at in enumerate(index(D))]


def load(cache, slots):
    """K, V [T, heads, D] at slots; zeros for -1."""
    T, H, D = len(slots), cache.shape[1], (cache.shape[3] - 16) // 32
    P = cache.shape[2] * 16
    out = np.zeros((2, T, H, D))
    blocks = {}
    for t, s in enumerate(map(int, slots)):
        if s >= 0:
            for h in range(H):
                key = (s // P, h, s % P // 16)
                if key not in blocks:
                    blocks[key] = load_block(cache[key])
                for n in range(2):
                    out[n, t, h] = blocks[key][n][s % 16]
    return out


def fork(held, table, parents, keep, ring, span, P, N):
    """The contract of kda_cache_fork in a loop.  Returns (kv, table, copies, span, ring,
    error)."""
    table, ring = np.array(table), np.array(ring)
    blocks = table.shape[1]
    err = False
    head, tail = map(int, span)
    if head < 0 or tail < head or tail - head > len(ring):
        head = tail = 0
        err = True
    avail, cap = tail - head, len(ring)
    pages_of = lambda n: -(-n // P)  # noqa: E731
    sound = [0 <= n and pages_of(n) <= blocks for n in held]
    err = err or not all(sound)
    before, kept = set(), set()
    for b, n in enumerate(held):
        for p in table[b, :pages_of(n)] if sound[b] else []:
            if 0 <= p < N:
                before.add(int(p))
            else:
                err = True
    out = np.full((len(parents), blocks), -1)
    kv, ends = [], {}
    for b, (p, n) in enumerate(zip(parents, keep)):
        ok = 0 <= p < len(held) and sound[p] and 0 <= n <= held[p]
        err = err or (p != -1 and not ok)
        kv.append(int(n) if ok else 0)
        out[b, :pages_of(kv[b])] = table[p, :pages_of(kv[b])] if ok else 0
        if kv[b] % P and 0 <= out[b, kv[b] // P] < N:
            ends.setdefault(int(out[b, kv[b] // P]), []).append(b)
    whole = {int(p) for b in range(len(parents)) for p in out[b, :kv[b] // P]}
    kept |= {p for p in whole if 0 <= p < N}
    copies = [[-1, -1, 0] for _ in parents]
    taken = 0
    for b in range(len(parents)):
        at = kv[b] // P
        p = int(out[b, at]) if kv[b] % P else -1
        if p not in ends:
            continue
        if p not in whole and ends[p][0] == b:
            kept.add(p)
        elif taken < avail:
            copies[b] = [p, int(ring[(head + taken) % cap]), kv[b] % P]
            out[b, at] = copies[b][1]
            taken += 1
        else:
            err = True
            out[b, at] = -1
            kv[b] -= kv[b] % P
    gone = sorted(before - kept)
    for i, p in enumerate(gone):
        ring[(tail + i) % cap] = p
    err = err or avail - taken + len(gone) > cap
    return kv, out, copies, (head + taken, tail + len(gone)), ring, err


def compact(held, table, ring, P, N):
    """The contract of kda_cache_compact.  Returns (table, copies, span, ring, error)."""
    table, ring = np.array(table), np.array(ring)
    blocks = table.shape[1]
    count = [-(-n // P) if n >= 0 and -(-n // P) <= blocks else None for n in held]
    err = None in count
    count = [c or 0 for c in count]
    entries = [int(p) for b, c in enumerate(count) for p in table[b, :c]]
    live = sorted({p for p in entries if 0 <= p < N})
    err = err or any(not 0 <= p < N for p in entries)
    L = len(live)
    src = [p for p in live if p >= L]
    dst = sorted(set(range(L)) - set(live))
    to = dict(zip(src, dst))
    out = np.full(table.shape, -1)
    for b, c in enumerate(count):
        out[b, :c] = [to.get(int(p), int(p)) for p in table[b, :c]]
    copies = [[a, b, P] for a, b in zip(src, dst)]
    copies += [[-1, -1, 0]] * (N // 2 - len(copies))
    ring[:N - L] = np.arange(L, N)
    return out, copies, (0, N - L), ring, err


def copy(cache, copies):
    """kda_cache_copy on one cache, in place."""
    for a, b, n in copies:
        if a >= 0:
            cache[b, :, :-(-n // 16)] = cache[a, :, :-(-n // 16)]
