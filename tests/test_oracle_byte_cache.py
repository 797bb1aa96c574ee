"""The fp64 oracle of the 8-bit cache and of shared pages pinned on the CPU: exponents and
ties, byte layout as a permutation, what a rising exponent does, invariants of the tables."""
import numpy as np
import pytest

from oracle import byte_cache as p8


def test_exponent():
    for top, want in [(448.0, 0), (449.0, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (0.0, -100),
                      (2.0 ** -300, -100), (3.4e38, 119), (448 * 2.0 ** 118, 118), (448 * 2.0 ** -100, -100),
                      (449 * 2.0 ** -100, -99)]:
        assert p8.exponent(top) == want, top


def test_code_ties_and_small_numbers():
    x = np.array([17.0, 19.0, 448.0, 460.0, np.inf, -np.inf, np.nan, 2.0 ** -10, 3 * 2.0 ** -10,
                  -(2.0 ** -9), 0.0, -1.0625, 1.1875])
    want = [16.0, 20.0, 448, 448, 448, -448, 0, 0, 2.0 ** -8, -(2.0 ** -9), 0, -1.0, 1.25]
    assert p8.value(p8.code(x, 0)).tolist() == want
    assert np.array_equal(p8.value(p8.code(x * 2.0 ** 33, 33), 33), np.array(want) * 2.0 ** 33)


@pytest.mark.parametrize("D", [64, 128])
def test_layout_is_a_permutation(D):
    k, v = p8.index(D)
    assert sorted(k.ravel()) == list(range(16 * D))
    assert sorted(v.ravel()) == list(range(16 * D, 32 * D))
    # runs that stay together: 16 channels of K, D / 8 of V
    assert (np.diff(k.reshape(16, D // 16, 16)) == 1).all()
    assert (np.diff(v.reshape(16, 8, D // 8)) == 1).all()


@pytest.mark.parametrize("D", [64, 128])
def test_store_load_and_a_rising_exponent(D):
    rng = np.random.RandomState(0)
    cache = np.zeros((3, 2, 2, 32 * D + 16), dtype=np.uint8)
    cache[..., :32 * D] = 0x7f  # NaN where nothing was stored
    k, v = rng.randn(2, 5, 2, D)
    slots = [32 + 16 + i for i in range(5)]
    p8.store(cache, slots, k, v)
    first = p8.load(cache, slots)
    assert np.abs(first[0] - k).max() <= np.abs(k).max() * 2.0 ** -4
    big = 64 * rng.randn(1, 2, D)
    p8.store(cache, [32 + 21], big, v[:1])
    both = p8.load(cache, slots + [32 + 21])
    # codes taken along: exact above 2^-6 2^e', else to a multiple of 2^-9 2^e'
    unit = 2.0 ** (cache[1, :, 1, 32 * D].astype(float) - 127)[:, None]
    keep = np.abs(first[0]) >= 2.0 ** -6 * unit
    assert np.array_equal(both[0][:5][keep], first[0][keep]) and not keep.all()
    assert np.abs(both[0][:5] - first[0]).max() <= (2.0 ** -10 * unit).max()
    assert np.array_equal(both[1][:5], first[1])
    # a token at a block's first place begins it anew
    p8.store(cache, [32 + 16], 2.0 ** -20 * k[:1], v[:1])
    again = p8.load(cache, [32 + 16])
    assert np.abs(again[0][0] - 2.0 ** -20 * k[0]).max() <= 2.0 ** -24 * np.abs(k[0]).max()


def _random_state(rng, B, P, blocks, N):
    """Rows that share pages: each continues the row before for some pages."""
    ids = list(rng.permutation(N))
    table, held = np.full((B, blocks), -1), []
    for b in range(B):
        n = rng.randint(0, min(blocks, 4) + 1)
        share = rng.randint(0, min(n, -(-held[-1] // P)) + 1) if b else 0
        for c in range(n):
            table[b, c] = table[b - 1, c] if c < share else ids.pop()
        held.append(n * P - rng.randint(0, P) if n else 0)
    cap = N + 3
    head = int(rng.randint(0, 50))
    ring = np.full(cap, -1)
    ring[(head + np.arange(len(ids))) % cap] = ids
    return held, table, ring, (head, head + len(ids))


def _holders(held, table, P):
    return [[int(p) for p in table[b, :-(-n // P)]] for b, n in enumerate(held)]


@pytest.mark.parametrize("seed", range(20))
def test_fork_keeps_what_rows_hold(seed):
    rng = np.random.RandomState(seed)
    P, N = 16, 60
    held, table, ring, span = _random_state(rng, 7, P, 5, N)
    R = rng.randint(0, 12)
    parents = rng.randint(-1, 7, R)
    keep = [int(rng.randint(0, held[p] + 1)) if p >= 0 else 0 for p in parents]
    content = {p: rng.randn(P) for p in range(N)}  # a page's tokens
    kv, out, copies, sp, rg, err = p8.fork(held, table, parents, keep, ring, span, P, N)
    assert not err and kv == keep
    after = {p: c.copy() for p, c in content.items()}
    for a, b, n in copies:
        if a >= 0:
            after[b][:n] = content[a][:n]
    rows = _holders(kv, out, P)
    for b, p in enumerate(parents):
        for t in range(kv[b]):
            assert after[rows[b][t // P]][t % P] == content[table[p, t // P]][t % P]
    # a page that a row ends inside is held by that row alone
    for b in range(R):
        if kv[b] % P:
            assert sum(rows[b][-1] in r for r in rows) == 1
    # every page is held or free, none both, none twice
    free = [int(rg[i % len(rg)]) for i in range(*sp)]
    used = {p for r in rows for p in r}
    assert sorted(free + list(used)) == list(range(N))


@pytest.mark.parametrize("seed", range(20))
def test_compact_keeps_what_rows_hold(seed):
    rng = np.random.RandomState(seed)
    P, N = 16, 60
    held, table, ring, _ = _random_state(rng, 9, P, 5, N)
    out, copies, span, rg, err = p8.compact(held, table, ring, P, N)
    assert not err and len(copies) == N // 2
    page = list(range(N))
    for a, b, n in copies:
        if a >= 0:
            page[b] = a
    for b, n in enumerate(held):
        for c in range(-(-n // P)):
            assert page[out[b, c]] == table[b, c]
    L = len({p for r in _holders(held, out, P) for p in r})
    assert {p for r in _holders(held, out, P) for p in r} == set(range(L))
    assert span == (0, N - L) and rg[:N - L].tolist() == list(range(L, N))
