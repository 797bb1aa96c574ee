"""The fp64 cache oracle pinned on the CPU: format tables, ties, byte layout as a
permutation, closed forms of attention, the page bookkeeping's invariants."""
import numpy as np
import pytest

from oracle import paged_cache as pc


def test_e4m3_values():
    assert pc.E4M3[1] == 2.0 ** -9 and pc.E4M3[8] == 2.0 ** -6 and pc.E4M3[-1] == 448.0
    assert np.all(np.diff(pc.E4M3) > 0) and np.isnan(pc.e4m3(0x7f))


def test_e2m1_ties_and_saturation():
    x = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -5.0, 0.26, 0.24,
                   -6.0, 5.01, 0.0]])
    codes, sb = pc.quantise(x)
    assert pc.e4m3(sb[0, 0]) == 1.0
    got = pc.dequantise(codes, sb)[0]
    assert got.tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 0, -1, -4, 0.5, 0, -6, 6, 0]


def test_scale_rounds_to_nearest_even_and_to_zero():
    for amax, want in [(6 * 1.0625, 1.0), (6 * 1.1875, 1.25), (6 * 500.0, 448.0),
                       (6 * 2.0 ** -10, 0.0), (6 * 1.01 * 2.0 ** -10, 2.0 ** -9)]:
        x = np.zeros((1, 16))
        x[0, 3] = amax
        codes, sb = pc.quantise(x)
        assert pc.e4m3(sb[0, 0]) == want, amax
        if want == 0:
            assert not codes.any()


@pytest.mark.parametrize("D", [64, 128])
def test_layout_is_a_permutation(D):
    kc, vc, ks, vs = pc._index(D)
    codes = sorted(set(kc.ravel()) | set(vc.ravel()))
    assert codes == list(range(16 * D))
    scales = sorted(set(ks.ravel()) | set(vs.ravel()))
    assert scales == list(range(16 * D, 18 * D))
    for at in (ks, vs):  # one byte for each token and block of 16 channels
        assert len(set(at[:, ::16].ravel())) == 16 * D // 16
        assert (at.reshape(16, D // 16, 16) == at[:, ::16, None]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_store_then_load(D):
    rng = np.random.RandomState(0)
    cache = rng.randint(0, 256, (3, 2, 2, 18 * D)).astype(np.uint8)
    before = cache.copy()
    k, v = rng.randn(2, D), rng.randn(2, D)
    pc.store(cache, [1 * 32 + 16 + 5], k[None], v[None])  # page 1, group 1, token 5
    for h in range(2):
        K, V = pc.load_group(cache[1, h, 1])
        assert np.array_equal(K[5], pc.dequantise(*pc.quantise(k[h])))
        assert np.array_equal(V[5], pc.dequantise(*pc.quantise(v[h])))
        K0, V0 = pc.load_group(before[1, h, 1])
        keep = np.arange(16) != 5
        assert np.array_equal(K[keep], K0[keep], equal_nan=True)
        assert np.array_equal(V[keep], V0[keep], equal_nan=True)
    same = np.ones((3, 2, 2), bool)
    same[1, :, 1] = False
    assert np.array_equal(cache[same], before[same])


def test_attention_closed_forms():
    rng = np.random.RandomState(1)
    q, k, v = rng.randn(1, 2, 64), rng.randn(5, 1, 64), rng.randn(5, 1, 64)
    out, lse, *_ = pc.attention(np.zeros_like(q), k, v, 1.0)
    assert np.allclose(out, v.mean(0)) and np.allclose(lse, np.log(5))
    out, lse, *_ = pc.attention(q, k[:1], v[:1], 0.3)
    assert np.allclose(out, v[0]) and np.allclose(lse[0, 1], 0.3 * q[0, 1] @ k[0, 0])
    # three new tokens over two cached ones: the first sees nothing
    out, lse, *_ = pc.attention(rng.randn(3, 1, 64), k[:2], v[:2], 1.0)
    assert not out[0].any() and lse[0, 0] == -np.inf and np.allclose(out[1, 0], v[0, 0])


def test_tables_conserve_pages():
    rng = np.random.RandomState(2)
    P, B, blocks, pages = 16, 9, 12, 70
    table = np.full((B, blocks), -1)
    ring, span = np.arange(pages), (0, pages)
    held = np.zeros(B, int)
    for step in range(60):
        seq = held - np.minimum(held, rng.randint(0, 20, B))
        new = rng.randint(-1, 40, B)
        kv, cu, slots, span, table, ring, err = pc.tables(held, seq, new, table, ring, span, P, 400)
        held = np.array(kv)
        owned = [table[b, j] for b in range(B) for j in range(-(-held[b] // P))]
        free = [ring[i % pages] for i in range(*span)]
        assert sorted(owned + free) == list(range(pages)), step
        live = [s for s in slots if s >= 0]
        assert len(set(live)) == len(live)
