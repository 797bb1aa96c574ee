"""GPU tests of the 4-bit paged cache against the fp64 oracle.

Tolerances.  Append, read and tables are exact.  Attention, per output element:
    |err| <= half step of the output type * |out|
             + sum_j p_j |v_j| * (w + 2 A 2^-17 + (L + 64) 2^-23)
             + (sum_j |v_j| / sum_j exp(s_j - max)) * 2^-24
w bounds the softmax weight's rounding before its product with v (half a step of
fp16, 2^-11, for bf16 outputs; 2^-21 for fp32 outputs, whose weights go in as two
halves); A = max_j scale sum_c |q_c k_jc| with D 2^-24 <= 2^-17 for a score's fp32
sum (an error d of a score moves the weights by a factor e^(2 d) at most); L keys
are summed in fp32; the last term is the weights too small for fp16's exponent.
The log-sum-exp: A 2^-16 + (L + 64) 2^-23 + |lse| 2^-22.
"""
import numpy as np
import pytest
import torch

import linear_attention_layer_gb300 as kda
from oracle import paged_cache as pc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    kda.get_device_error()
    yield
    assert kda.get_device_error() == 0


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------ append, read ---

def _values(rng, shape):
    """Unequal channels, zero and tiny and huge blocks, exact ties of code and scale."""
    x = rng.randn(*shape) * np.exp2(rng.randint(-3, 4, shape[-2:]))
    t = x.reshape(-1, 16)
    n = len(t)
    t[rng.permutation(n)[: n // 8]] = 0
    t[rng.permutation(n)[: n // 16]] *= 2.0 ** -14
    t[rng.permutation(n)[: n // 16]] *= 2.0 ** 9
    ties = rng.permutation(n)[: n // 8]
    t[ties] = rng.choice(np.concatenate([pc.E2M1, (pc.E2M1[1:] + pc.E2M1[:-1]) / 2]), (len(ties), 16))
    t[ties, 0] = 6 * rng.choice([1.0, 1.0625, 1.125, 1.1875], len(ties))  # scale ties too
    return x


def _exact(x):
    return pc.dequantise(*pc.quantise(x.double().cpu().numpy()))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,H,P,T", [(128, 8, 64, 37), (64, 3, 16, 33), (128, 1, 48, 1),
                                     (64, 2, 256, 300), (128, 5, 32, 16)])
@pytest.mark.parametrize("layout", ["packed", "slices", "odd"])
def test_append_read(dtype, D, H, P, T, layout):
    rng = np.random.RandomState(D + H + T)
    pages = -(-T // P) + 3
    slots = rng.permutation(pages * P)[:T]
    slots[T // 2: T // 2 + 1] = -1
    src = torch.tensor(_values(rng, (T, 2 * H, D)), device=DEV).to(dtype)
    if layout == "packed":
        k, v = src[:, :H].contiguous(), src[:, H:].contiguous()
    elif layout == "slices":
        k, v = src[:, :H], src[:, H:]
    else:  # rows that start off a 16-byte boundary
        wide = torch.zeros((T, 2 * H, D + 3), dtype=dtype, device=DEV)
        wide[..., 1:D + 1] = src
        k, v = wide[:, :H, 1:D + 1], wide[:, H:, 1:D + 1]
    cache = torch.tensor(rng.randint(0, 256, (pages, H, P // 16, 18 * D)).astype(np.uint8),
                         device=DEV)
    want = cache.cpu().numpy().copy()
    live = slots >= 0
    pc.store(want, slots[live], k.double().cpu().numpy()[live], v.double().cpu().numpy()[live])
    st = torch.tensor(slots, device=DEV)
    kda.cache_append(k, v, st, cache)
    got = cache.cpu().numpy()
    # codes of -0 and +0 stand for the same value: compare values, and bytes not written
    for p in range(pages):
        for h in range(H):
            for g in range(P // 16):
                a, b = pc.load_group(got[p, h, g]), pc.load_group(want[p, h, g])
                assert np.array_equal(a[0], b[0], equal_nan=True)
                assert np.array_equal(a[1], b[1], equal_nan=True)
    kr, vr = kda.cache_read(st, cache, dtype)
    for x, r in ((k, kr), (v, vr)):
        e = _exact(x)
        e[~live] = 0
        assert np.array_equal(r.double().cpu().numpy(), e)


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_exponents(dtype):
    rng = np.random.RandomState(5)
    T, H, D = 20, 3, 64
    ke, ve = [-9, 0, 7], [3, -20, 64]
    x = torch.tensor(rng.randn(2, T, H, D), device=DEV)
    k = (x[0] * torch.exp2(torch.tensor(ke, device=DEV).double())[:, None]).to(dtype)
    v = (x[1] * torch.exp2(torch.tensor(ve, device=DEV).double())[:, None]).to(dtype)
    cache = kda.cache_empty(2, 16, H, D, DEV)
    slots = torch.arange(T, device=DEV)
    kda.cache_append(k, v, slots, cache, k_exponent=i32(ke), v_exponent=i32(ve))
    kr, vr = kda.cache_read(slots, cache, dtype, k_exponent=i32(ke), v_exponent=i32(ve))
    for x, r, e in ((k, kr, ke), (v, vr, ve)):
        s = np.exp2(np.array(e, float))[:, None]
        want = pc.dequantise(*pc.quantise(x.double().cpu().numpy() / s)) * s
        assert np.array_equal(r.double().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_non_finite(dtype):
    D = 64
    k = torch.ones((2, 1, D), dtype=dtype, device=DEV)
    v = torch.ones_like(k)
    k[0, 0, 3], k[0, 0, 20], v[1, 0, 40] = float("nan"), float("inf"), float("-inf")
    cache = kda.cache_empty(1, 16, 1, D, DEV)
    slots = torch.arange(2, device=DEV)
    kda.cache_append(k, v, slots, cache)
    assert kda.get_device_error() == 5
    kr, vr = (x.float().cpu().numpy() for x in kda.cache_read(slots, cache, dtype))
    one = float(pc.dequantise(*pc.quantise(np.ones((1, 16))))[0, 0])  # of a block of ones
    assert kr[0, 0, 3] == 0 and kr[0, 0, 2] == one
    assert kr[0, 0, 20] == 2688 and kr[0, 0, 21] == 0 and vr[1, 0, 40] == -2688
    assert (kr[1] == one).all() and (vr[0] == one).all()


def test_bad_slots_are_skipped():
    cache = torch.full((2, 1, 1, 18 * 64), 7, dtype=torch.uint8, device=DEV)
    x = torch.randn((3, 1, 64), device=DEV)
    for bad in (32, -2, 1 << 40):
        slots = torch.tensor([bad, -1, bad], device=DEV)
        kda.cache_append(x, x, slots, cache)
        assert kda.get_device_error() == 5
        assert (cache == 7).all()
        k, v = kda.cache_read(slots, cache, torch.float32)
        assert kda.get_device_error() == 5
        assert not k.any() and not v.any()


# ------------------------------------------------------------------ tables ---

def _tables(held, seq, new, table, ring, span, P, cap, **kw):
    t, r = i32(table), i32(ring)
    out = kda.cache_tables(i32(held), i32(seq), i32(new), t, r,
                           torch.tensor(span, dtype=torch.int64, device=DEV), page_size=P,
                           max_tokens=cap, **kw)
    return [x.cpu().numpy() for x in (*out, t, r)]


def _check_tables(held, seq, new, table, ring, span, P, cap):
    got = _tables(held, seq, new, table, ring, span, P, cap)
    kv, cu, slots, sp, tb, rg, err = pc.tables(held, seq, new, table, ring, span, P, cap)
    for g, w in zip(got, (kv, cu, slots, sp, tb, rg)):
        assert np.array_equal(g, w)
    assert kda.get_device_error() == (5 if err else 0)
    return np.array(kv, dtype=np.int64), sp, tb, rg


@pytest.mark.parametrize("B,P,steps,most", [(1, 16, 6, 40), (37, 16, 6, 9), (300, 64, 4, 3),
                                            (64, 64, 2, 900), (1500, 32, 3, 2)])
def test_tables_follow_lengths(B, P, steps, most):
    rng = np.random.RandomState(B)
    blocks = steps * most // P + 3
    pages = B * blocks // 2 + 2
    table = np.full((B, blocks), -1)
    span = (5 * pages - 3, 6 * pages - 3)
    ring = rng.permutation(pages)
    held = np.zeros(B, int)
    for _ in range(steps):
        seq = held - np.minimum(held, rng.randint(0, 5, B))
        new = rng.randint(-1, most + 1, B)
        held, span, table, ring = _check_tables(held, seq, new, table, ring, span, P,
                                                int(np.maximum(new, 0).sum()) + rng.randint(0, 5))


def test_tables_refusals():
    P, ring = 16, np.arange(4)
    table = np.full((5, 3), -1)
    table[2, 0] = 9
    # rows too short, ring empty for the third and after, one that needs none goes through
    _check_tables([0, 0, 16, 0, 0], [0, 0, 7, 0, 0], [49, 40, 40, 1, 0], table, ring, (0, 4), P, 200)
    _check_tables([0, 0, 16, 0, 0], [0, 0, 7, 0, 0], [0, 40, 9, 20, 0], table, ring, (0, 4), P, 200)
    # malformed lengths
    for held, seq, new in [([-1], [0], [2]), ([4], [5], [1]), ([4], [-1], [1]), ([4], [4], [-2]),
                           ([49], [1], [1]), ([4], [4], [2 ** 31 - 1])]:
        _check_tables(held, seq, new, table[:1], ring, (0, 4), P, 7)
    # malformed ring
    for span in [(-1, 2), (3, 2), (0, 5)]:
        _check_tables([0], [0], [3], table[:1], ring, span, P, 8)
        _check_tables([30], [0], [-1], np.array([[1, 2, -1]]), ring, span, P, 8)
    # more tokens than slots, none at all, no requests
    _check_tables([0, 0], [0, 0], [9, 9], table[:2], ring, (0, 4), P, 11)
    _check_tables([3, 0], [3, 0], [0, 0], np.array([[1, 0, 0], [0, 0, 0]]), ring, (2, 4), P, 0)
    _check_tables([], [], [], np.zeros((0, 3), int), ring, (2, 4), P, 6)


def test_tables_in_place_loop_in_a_graph():
    P, B, pages = 16, 6, 40
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    new = i32([1, 2, 3, 0, 1, 4])
    table = torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    ring = torch.arange(pages, dtype=torch.int32, device=DEV)
    span = torch.tensor([0, pages], device=DEV)
    cu, slots = i32(np.zeros(B + 1)), torch.zeros(16, dtype=torch.int64, device=DEV)

    def step():
        kda.cache_tables(lens, lens, new, table, ring, span, page_size=P, max_tokens=16,
                         kv_lens=lens, cu_new=cu, slots=slots, free_range_out=span)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(9):
        g.replay()
    torch.cuda.synchronize()
    held, t, r, sp = np.zeros(B, int), np.full((B, 8), -1), np.arange(pages), (0, pages)
    for _ in range(10):
        held, _, s, sp, t, r, _ = pc.tables(held, held, [1, 2, 3, 0, 1, 4], t, r, sp, P, 16)
    assert lens.tolist() == held and slots.tolist() == s and span.tolist() == list(sp)
    assert np.array_equal(table.cpu().numpy(), t) and np.array_equal(ring.cpu().numpy(), r)


# --------------------------------------------------------------- attention ---

class Problem:
    """Requests over a cache of random pages; the bytes no request holds are random too,
    scales of NaN among them."""

    def __init__(self, kv, new, Hq, Hk, D, P, dtype, seed=0, extra_pages=2, qscale=1.5):
        rng = np.random.RandomState(seed)
        self.kv, self.new, self.Hq, self.Hk, self.D, self.P = kv, new, Hq, Hk, D, P
        need = [-(-n // P) for n in kv]
        pages = sum(need) + extra_pages
        ids = rng.permutation(pages)
        self.table = np.full((len(kv), max(need + [1])), -7)
        raw = rng.randint(0, 256, (pages, Hk, P // 16, 18 * D)).astype(np.uint8)
        raw[..., 16 * D:][rng.rand(*raw.shape[:3], 2 * D) < 0.2] = 0x7f
        self.ks, self.vs = [], []
        at = 0
        for b, n in enumerate(kv):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            k = rng.randn(n, Hk, D) * np.exp2(rng.randint(-2, 2, (Hk, D)))
            v = rng.randn(n, Hk, D)
            if n:
                pos = np.arange(n)
                pc.store(raw, self.table[b, pos // P] * P + pos % P, k, v)
            self.ks.append(pc.dequantise(*pc.quantise(k)) if n else k)
            self.vs.append(pc.dequantise(*pc.quantise(v)) if n else v)
        self.cache = torch.tensor(raw, device=DEV)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(int)
        self.q = torch.tensor(rng.randn(self.cu[-1], Hq, D) * qscale, device=DEV).to(dtype)

    def call(self, **kw):
        q = kw.pop("q", self.q)
        kw.setdefault("max_new", max(self.new + [1]))
        return kda.cache_attention(q, kw.pop("cache", self.cache), i32(kw.pop("table", self.table)),
                                   i32(kw.pop("kv", self.kv)), i32(kw.pop("cu", self.cu)),
                                   return_lse=True, **kw)

    def check(self, out, lse, scale=None, only=None, kf=1.0, vf=1.0):
        scale = self.D ** -0.5 if scale is None else scale
        q = self.q.double().cpu().numpy()
        out_h, lse_h = out.double().cpu().numpy(), lse.double().cpu().numpy()
        bf16 = self.q.dtype == torch.bfloat16
        for b, (L, n) in enumerate(zip(self.kv, self.new)):
            if only is not None and b not in only:
                continue
            rows = slice(self.cu[b], self.cu[b + 1])
            o, z, mass, flat, size = pc.attention(q[rows], self.ks[b] * kf, self.vs[b] * vf, scale)
            A = size[..., None]
            tol = (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(o) + mass * (
                (2.0 ** -11 if bf16 else 2.0 ** -21) + A * 2.0 ** -16 + (L + 64) * 2.0 ** -23) + \
                flat * 2.0 ** -24
            err = np.abs(out_h[rows] - o)
            assert np.isfinite(out_h[rows]).all(), f"request {b}"
            bad = err > tol
            assert not bad.any(), (b, L, n, float((err / np.maximum(tol, 1e-300)).max()))
            empty = np.isinf(z)
            assert np.array_equal(np.isinf(lse_h[rows]), empty) and (lse_h[rows][empty] < 0).all()
            ltol = size * 2.0 ** -16 + (L + 64) * 2.0 ** -23 + np.abs(np.where(empty, 0, z)) * 2.0 ** -22
            assert (np.abs(np.where(empty, 0, lse_h[rows] - np.where(empty, 0, z))) <= ltol).all(), b


RAGGED = [1, 0, 15, 16, 17, 63, 64, 65, 129, 200, 333]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,Hk,P", [(128, 8, 2, 64), (64, 3, 3, 16), (128, 1, 1, 48),
                                       (64, 16, 1, 32), (128, 10, 2, 16), (128, 24, 1, 128),
                                       (64, 40, 1, 64)])
def test_decode(dtype, D, Hq, Hk, P):
    p = Problem(RAGGED, [1] * len(RAGGED), Hq, Hk, D, P, dtype, seed=D + Hq)
    p.check(*p.call())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,Hk,P", [(128, 8, 2, 64), (64, 6, 3, 16), (128, 16, 1, 32)])
def test_windows(dtype, D, Hq, Hk, P):
    kv = [5, 0, 3, 16, 18, 70, 130, 64, 90, 7]
    new = [5, 0, 4, 3, 2, 7, 1, 8, 0, 9]  # some longer than their context: empty rows
    p = Problem(kv, new, Hq, Hk, D, P, dtype, seed=Hq)
    p.check(*p.call())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,Hk,P,kv,new", [
    (128, 8, 2, 64, [300, 129], [130, 129]), (64, 4, 4, 16, [257], [257]),
    (128, 4, 1, 32, [64, 700, 33], [64, 65, 40]), (128, 16, 2, 256, [513], [33]),
    (64, 12, 2, 64, [100, 50, 260, 0], [1, 50, 129, 3])])
def test_chunks(dtype, D, Hq, Hk, P, kv, new):
    p = Problem(kv, new, Hq, Hk, D, P, dtype, seed=sum(new))
    p.check(*p.call())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,new", [([40, 700], [100, 300]), ([2000], [90]), ([257, 5, 64], [256, 5, 60])])
def test_chunks_of_many_rows(D, kv, new):
    """More rows than a unit has, contexts shorter than the chunk, contexts cut over CTAs."""
    p = Problem(kv, new, 8, 1, D, 48, torch.bfloat16, seed=D + sum(kv))
    p.check(*p.call())


@pytest.mark.parametrize("rows", [8, 9, 16, 17, 47, 48, 49, 128, 129, 256, 257])
def test_row_counts_at_the_kernels_borders(rows):
    p = Problem([300, 310], [rows, 1], 1, 1, 64, 16, torch.bfloat16, seed=rows)
    p.check(*p.call())


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_long_request(dtype):
    p = Problem([4100], [2], 4, 2, 128, 64, dtype, seed=3)
    p.check(*p.call())


def test_many_requests():
    rng = np.random.RandomState(8)
    kv = list(map(int, rng.randint(0, 90, 2100)))
    p = Problem(kv, [1] * len(kv), 2, 1, 64, 16, torch.bfloat16, seed=8)
    p.check(*p.call(), only=set(range(0, 2100, 37)) | {2047, 2048, 2049, 2099})


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 3, 40])
def test_strided_and_odd_queries(dtype, new):
    p = Problem([70, 200], [new, new], 4, 2, 128, 32, dtype, seed=2)
    base = p.call()
    T = p.q.shape[0]
    wide = torch.full((T, 3, 4, 128), 9.0, dtype=dtype, device=DEV)
    wide[:, 1] = p.q
    for q in (wide[:, 1],):
        for a, b in zip(base, p.call(q=q)):
            assert torch.equal(a, b)
    odd = torch.full((T, 4, 131), 9.0, dtype=dtype, device=DEV)
    odd[..., 1:129] = p.q
    for a, b in zip(base, p.call(q=odd[..., 1:129])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("new", [1, 40])
def test_scale_exponents_and_large_scores(new):
    ke, ve = [4, -30], [-3, 12]
    p = Problem([150, 77], [new, new], 4, 2, 64, 32, torch.float32, seed=9)
    kf, vf = (np.exp2(np.array(e, float))[:, None] for e in (ke, ve))
    out = p.call(scale=0.07, k_exponent=i32(ke), v_exponent=i32(ve))
    p.check(*out, scale=0.07, kf=kf, vf=vf)
    # scores of hundreds: one key takes all
    p = Problem([150, 77], [new, new], 4, 2, 64, 32, torch.bfloat16, seed=9, qscale=200.0)
    p.check(*p.call(scale=1.0), scale=1.0)
    p = Problem([150, 77], [new, new], 4, 2, 64, 32, torch.bfloat16, seed=9)
    p.check(*p.call(scale=0.0), scale=0.0)
    p.check(*p.call(scale=-0.2), scale=-0.2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mag", [1e-30, 1e30])
def test_queries_of_any_magnitude(dtype, mag):
    p = Problem([90], [2], 4, 2, 128, 32, dtype, seed=4)
    p.q = (p.q.double() * mag).to(dtype)
    scale = 0.1 / mag
    p.check(*p.call(scale=scale), scale=np.float64(np.float32(scale)))


@pytest.mark.parametrize("new", [1, 40])
def test_non_finite_query_stays_in_its_row(new):
    p = Problem([90, 64], [new, new], 4, 2, 128, 32, torch.bfloat16, seed=4)
    base, base_lse = p.call()
    q = p.q.clone()
    q[0, 1, 5] = float("nan")
    q[new, 3, 0] = float("inf")
    out, lse = p.call(q=q)
    assert out[0, 1].isnan().all() and lse[0, 1].isnan()
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device=DEV)
    keep[0, 1] = keep[new, 3] = False
    assert torch.equal(out[keep], base[keep]) and torch.equal(lse[keep], base_lse[keep])


@pytest.mark.parametrize("new", [1, 40])
def test_bad_tables_and_lengths(new):
    p = Problem([100, 100, 100], [new] * 3, 4, 2, 128, 32, torch.bfloat16, seed=6)
    base, base_lse = p.call()
    for page in (-1, 1 << 20):
        t = p.table.copy()
        t[1, 1] = page
        out, lse = p.call(table=t)
        assert kda.get_device_error() == 5
        for b in (0, 2):
            assert torch.equal(out[p.cu[b]:p.cu[b + 1]], base[p.cu[b]:p.cu[b + 1]])
        hidden = Problem([100, 100, 100], [new] * 3, 4, 2, 128, 32, torch.bfloat16, seed=6)
        keep = np.r_[0:32, 64:100]
        hidden.ks[1], hidden.vs[1] = hidden.ks[1][keep], hidden.vs[1][keep]
        hidden.kv = [100, 68, 100]
        if new == 1:
            hidden.check(out, lse, only={1})
        assert out.isfinite().all()
    for kv in ([100, -5, 100], [100, 4 * 32 + 1, 100]):
        out, lse = p.call(kv=kv, out=torch.full_like(base, 3.0))
        assert kda.get_device_error() == 5
        assert torch.equal(out[:p.cu[1]], base[:p.cu[1]])
        assert torch.equal(out[p.cu[2]:], base[p.cu[2]:])
        assert (out[p.cu[1]:p.cu[2]] == 3.0).all()
    cu = p.cu.copy()
    cu[2] = cu[1] - 1  # not monotone: requests 1 and 2 are touched by it
    out, lse = p.call(cu=cu)
    assert kda.get_device_error() == 5
    assert torch.equal(out[:new], base[:new])
    cu = p.cu.copy()
    cu[3] += 1  # past the packed batch
    out, lse = p.call(cu=cu)
    assert kda.get_device_error() == 5
    assert torch.equal(out[:2 * new], base[:2 * new])


@pytest.mark.parametrize("new,hint", [(1, 1), (3, 40), (40, 1), (200, 7)])
def test_max_new_is_a_hint(new, hint):
    p = Problem([300, 90], [new, min(new, 5)], 8, 2, 128, 32, torch.bfloat16, seed=6)
    p.check(*p.call(max_new=hint))


def test_padding_tokens_are_left_alone():
    p = Problem([40, 70], [1, 1], 4, 2, 64, 16, torch.bfloat16)
    q = torch.cat([p.q, p.q.new_full((3, 4, 64), float("nan"))])
    out = torch.full_like(q, 5.0)
    o, _ = p.call(q=q, out=out)
    assert (o[2:] == 5.0).all()
    p.check(o[:2], _[:2])


def test_no_heads_share_and_empty_batch():
    p = Problem([0, 0], [1, 4], 4, 2, 64, 16, torch.float32)
    p.check(*p.call())
    p = Problem([9, 0], [0, 0], 4, 2, 64, 16, torch.float32)
    out, lse = p.call()
    assert out.shape == (0, 4, 64)


def test_pages_beyond_32_bits():
    """A cache of more than 2^32 bytes, the request's pages at its end."""
    Hk, D, P = 8, 128, 256
    pages = (1 << 32) // (Hk * P // 16 * 18 * D) + 40
    small = Problem([700], [1], 8, Hk, D, P, torch.bfloat16, seed=1, extra_pages=0)
    cache = torch.empty((pages, Hk, P // 16, 18 * D), dtype=torch.uint8, device=DEV)
    n = small.cache.shape[0]
    cache[-n:] = small.cache
    table = np.where(small.table >= 0, small.table + pages - n, -1)
    small.check(*small.call(cache=cache, table=table))
    slots = torch.tensor([(pages - 1) * P + 3, (pages - 40) * P], device=DEV)
    x = torch.randn((2, Hk, D), device=DEV)
    kda.cache_append(x, -x, slots, cache)
    k, v = kda.cache_read(slots, cache, torch.float32)
    assert np.array_equal(k.double().cpu().numpy(), _exact(x)) and torch.equal(k, -v)


@pytest.mark.parametrize("new", [1, 3, 70])
def test_graph_and_side_stream(new):
    p = Problem([150, 90, 400], [new, 0, new], 8, 2, 128, 32, torch.bfloat16, seed=12)
    base = p.call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = p.call(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(base, side))
    table, kv, cu = i32(p.table), i32(p.kv), i32(p.cu)
    out = torch.zeros_like(p.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.cache_attention(p.q, p.cache, table, kv, cu, max_new=new, out=out)
    kv2 = [120, 90, 333]
    kv.copy_(i32(kv2))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, p.call(kv=kv2)[0])


def test_repeatable():
    p = Problem([3000, 70, 800], [4, 1, 2], 8, 2, 128, 32, torch.bfloat16, seed=12)
    a = p.call()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, p.call()))


def test_append_then_attend():
    """The step a server makes: tables, append, attention, over three steps."""
    P, B, Hk, Hq, D = 16, 3, 2, 8, 64
    rng = np.random.RandomState(3)
    cache = kda.cache_empty(30, P, Hk, D, DEV)
    table = torch.full((B, 6), -1, dtype=torch.int32, device=DEV)
    ring = torch.arange(30, dtype=torch.int32, device=DEV)
    span = torch.tensor([0, 30], device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    p = Problem([], [], Hq, Hk, D, P, torch.bfloat16)
    p.ks = p.vs = None
    ks = [np.zeros((0, Hk, D))] * B
    vs = [np.zeros((0, Hk, D))] * B
    for new in ([20, 33, 5], [1, 1, 1], [3, 0, 2]):
        T = sum(new)
        k, v = (torch.tensor(rng.randn(T, Hk, D), device=DEV).bfloat16() for _ in range(2))
        p.q = torch.tensor(rng.randn(T, Hq, D), device=DEV).bfloat16()
        lens, cu, slots, span = kda.cache_tables(lens, lens, i32(new), table, ring, span,
                                                 page_size=P, max_tokens=T)
        kda.cache_append(k, v, slots, cache)
        out, lse = kda.cache_attention(p.q, cache, table, lens, cu, max_new=max(new),
                                       return_lse=True)
        p.cu = np.concatenate([[0], np.cumsum(new)]).astype(int)
        for b in range(B):
            rows = slice(p.cu[b], p.cu[b + 1])
            ks[b] = np.concatenate([ks[b], _exact(k[rows])])
            vs[b] = np.concatenate([vs[b], _exact(v[rows])])
        p.ks, p.vs, p.new = ks, vs, new
        p.kv = [len(x) for x in ks]
        assert lens.tolist() == p.kv
        p.check(out, lse)
