"""The bf16 rounding of the cache's append, restated step by step in fp32 and compared with the
exact one for every bf16 value and every scale.

The kernel does not divide: it takes x times an approximate reciprocal of the scale s, at most
2 units in the last place off, and brings the product back onto the borders between codes by
rounding it to a multiple of 2^-12 (one fused addition of 2560, which is taken away again).  The
scale is max |x| times a rounded 1/6, rounded to 16 fraction bits, before E4M3's own rounding."""
import numpy as np
import pytest

from oracle import paged_cache as pc

F32 = np.float32
BITS = np.arange(0x7f80, dtype=np.uint32) << 16
EVERY = BITS.view(np.float32)  # the non-negative finite bf16 values
WIDE = EVERY.astype(np.float64)


def _scales():
    """Scale byte of a block with each value as its largest: (restated, exact)."""
    top = np.minimum(EVERY, F32(3e38)) * (F32(1) / F32(6))
    rounded = ((top.view(np.uint32) + np.uint32(0x40)) & ~np.uint32(0x7f)).view(np.float32)
    return pc.nearest(pc.E4M3, rounded.astype(np.float64)), _exact_scale(WIDE)


def _exact_scale(x):
    """nearest(E4M3, x / 6) without the division: x against 6 times the borders, both exact."""
    mids = 6 * (pc.E4M3[1:] + pc.E4M3[:-1]) / 2
    idx = np.searchsorted(mids, x, side="left")          # borders below x
    tie = (idx < len(mids)) & (x == mids[np.minimum(idx, len(mids) - 1)])
    return idx + (tie & (idx % 2 == 1))


def test_every_scale():
    got, want = _scales()
    assert np.array_equal(got, want)


def _codes(x, s, r):
    """Codes of x (fp32) with r for 1 / s: the product and 2560 added with one rounding."""
    y = (x.astype(np.float64) * np.float64(r) + 2560.0).astype(np.float32) - F32(2560)
    return pc.nearest(pc.E2M1, y.astype(np.float64))


@pytest.mark.parametrize("ulps", [-2, -1, 0, 1, 2])
def test_every_code(ulps):
    """All values that a block of the scale can hold: up to the largest that gives it."""
    scale = _exact_scale(WIDE)
    mids = (pc.E2M1[1:] + pc.E2M1[:-1]) / 2
    for sb in range(1, 127):
        s = pc.E4M3[sb]
        x = EVERY[WIDE <= WIDE[scale == sb].max()]
        r = F32(1) / F32(s)
        r = (np.array([r]).view(np.int32) + np.int32(ulps)).view(np.float32)[0]
        wide = x.astype(np.float64)
        want = sum(((wide > m * s) | ((wide == m * s) & (i % 2 == 1))).astype(int)
                   for i, m in enumerate(mids))
        assert np.array_equal(_codes(x, s, r), want), sb


def test_a_planted_slip_is_seen():
    """Without the rounding onto the borders a reciprocal off by one unit moves ties."""
    sb = 0x36  # 0.875: 1 / s is not exact
    s = pc.E4M3[sb]
    tie = np.array([2.5 * s], F32)
    assert WIDE[_exact_scale(WIDE) == sb].max() > tie[0]
    r = (np.array([F32(1) / F32(s)]).view(np.int32) + np.int32(2)).view(np.float32)[0]
    raw = (tie.astype(np.float64) * np.float64(r)).astype(np.float32)
    assert pc.nearest(pc.E2M1, raw.astype(np.float64))[0] != _codes(tie, s, r)[0] == 4
