"""GPU tests of the 8-bit paged cache against the fp64 oracle.

Append and read are exact.  Attention, per output element, as for the 4-bit cache
(tests/test_gpu_cache.py has the terms), the weights too small for fp16's exponent
measured under the request's largest exponent of V:
    |err| <= half step of the output type * |out|
             + sum_j p_j |v_j| * (w + 2 A 2^-17 + (L + 64) 2^-23)
             + (sum_j |v_j| 2^(E - e_j) / sum_j exp(s_j - max)) * 2^-31
A weight's place below the largest is at most 2^-32 off (half a step of fp16's
smallest numbers, 2^-25, under a reference that leaves the largest 2^7 at least).
"""
import numpy as np
import pytest
import torch

import linear_attention_layer_gb300 as kda
from oracle import paged_cache as pc
from oracle import byte_cache as p8
from tests.test_gpu_cache import DEV, DTYPES, RAGGED, _device, i32  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ append, read ---

def _values(rng, shape):
    """Unequal channels, tokens of zeros, tiny and huge ones, ties of codes, largest values on a
    border between two exponents."""
    x = rng.randn(*shape) * np.exp2(rng.randint(-3, 4, shape[-2:]))
    t = x.reshape(-1, shape[-1])
    n = len(t)
    t[rng.permutation(n)[: n // 8]] = 0
    t[rng.permutation(n)[: n // 8]] *= 2.0 ** -14
    t[rng.permutation(n)[: n // 8]] *= 2.0 ** 9
    ties = rng.permutation(n)[: n // 4]
    mids = (pc.E4M3[1:] + pc.E4M3[:-1]) / 2
    t[ties] = rng.choice(np.concatenate([pc.E4M3, mids]), (len(ties), shape[-1]))
    t[ties, 0] = rng.choice([448.0, 450.0, 446.0], len(ties))
    return x


def _slots(rng, T, P, pages, order):
    """Slots of T tokens, those of a block next to one another."""
    if order == "runs":  # requests of any length, each from any place of a page of its own
        slots, page, ids = [], 0, rng.permutation(pages)
        while len(slots) < T:
            n = min(T - len(slots), int(rng.randint(1, 2 * P)))
            pos = rng.randint(0, P) + np.arange(n)
            if page + pos[-1] // P >= pages:
                break
            slots += [int(ids[page + p // P]) * P + int(p) % P for p in pos]
            page += pos[-1] // P + 1
        slots += [-1] * (T - len(slots))
        if T > 20:  # skipped: one in between and what its block would still get
            block = slots[T // 2] // 16
            slots = [-1 if i >= T // 2 and s // 16 == block else s for i, s in enumerate(slots)]
        return slots
    blocks = rng.permutation(pages * P // 16)[:T]  # one token of each block
    return [int(b) * 16 + int(rng.randint(0, 16)) for b in blocks]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,H,P,T", [(128, 8, 64, 37), (64, 3, 16, 33), (128, 1, 48, 1),
                                     (64, 2, 256, 300), (128, 5, 32, 16)])
@pytest.mark.parametrize("layout", ["packed", "slices", "odd"])
@pytest.mark.parametrize("order", ["runs", "scattered"])
def test_append_read(dtype, D, H, P, T, layout, order):
    rng = np.random.RandomState(D + H + T)
    pages = max(-(-T // P) * 2 + 5, -(-T * 16 // P) + 1)
    slots = _slots(rng, T, P, pages, order)
    src = torch.tensor(_values(rng, (T, 2 * H, D)), device=DEV).to(dtype)
    if layout == "packed":
        k, v = src[:, :H].contiguous(), src[:, H:].contiguous()
    elif layout == "slices":
        k, v = src[:, :H], src[:, H:]
    else:  # rows that start off a 16-byte boundary
        wide = torch.zeros((T, 2 * H, D + 3), dtype=dtype, device=DEV)
        wide[..., 1:D + 1] = src
        k, v = wide[:, :H, 1:D + 1], wide[:, H:, 1:D + 1]
    raw = rng.randint(0, 256, (pages, H, P // 16, 32 * D + 16)).astype(np.uint8)
    raw[..., 32 * D:32 * D + 2] = rng.randint(110, 130, raw.shape[:3] + (2,))
    cache = torch.tensor(raw, device=DEV)
    p8.store(raw, slots, k.double().cpu().numpy(), v.double().cpu().numpy())
    st = torch.tensor(slots, device=DEV)
    kda.byte_cache_append(k, v, st, cache)
    got = cache.cpu().numpy()
    # NaN codes of either sign that were there stand for the same: values and exponents
    assert np.array_equal(got[..., 32 * D:], raw[..., 32 * D:])
    assert np.array_equal(p8.value(got[..., :32 * D]), p8.value(raw[..., :32 * D]), equal_nan=True)
    for x, r in zip(p8.load(raw, slots), kda.byte_cache_read(st, cache, dtype)):
        assert np.array_equal(r.double().cpu().numpy(), x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_append_in_long_batches(dtype, D):
    """Batches long enough for the form that takes 16 tokens a warp: prompts from any place,
    single tokens between them, slots of -1."""
    rng = np.random.RandomState(D)
    H, P, T = 24, 32, 5600
    pages = 400
    ids, page, slots = rng.permutation(pages), 0, []
    while len(slots) < T:
        n = min(T - len(slots), int(rng.choice([1, 1, 2, 15, 16, 17, 40, 300])))
        pos = rng.randint(0, P) + np.arange(n)
        slots += [int(ids[page + p // P]) * P + int(p) % P for p in pos]
        page += pos[-1] // P + 1
        if rng.rand() < 0.1:
            slots += [-1] * int(rng.randint(1, 20))
    slots = slots[:T]
    src = torch.tensor(_values(rng, (T, 2 * H, D)), device=DEV).to(dtype)
    cache = torch.randint(0, 120, (pages, H, P // 16, 32 * D + 16), dtype=torch.uint8, device=DEV)
    cache[..., 32 * D:32 * D + 2] = 120
    some = [0, 11, 23]  # heads that are compared
    raw = cache[:, some].cpu().numpy()
    x = src.double().cpu().numpy()
    p8.store(raw, slots, x[:, some], x[:, [H + h for h in some]])
    kda.byte_cache_append(src[:, :H], src[:, H:], torch.tensor(slots, device=DEV), cache)
    got = cache[:, some].cpu().numpy()
    assert np.array_equal(got[..., 32 * D:], raw[..., 32 * D:])
    assert np.array_equal(p8.value(got[..., :32 * D]), p8.value(raw[..., :32 * D]))


@pytest.mark.parametrize("D", [64, 128])
def test_tokens_one_at_a_time(D):
    """A block that grows token by token, in windows, and is begun anew: the exponent rises and
    what is there is taken along, each step as the oracle has it."""
    rng = np.random.RandomState(3)
    H, T = 2, 40
    x = rng.randn(2, T, H, D) * np.exp2(rng.randint(-12, 13, (2, T, H, 1)))
    k, v = (torch.tensor(y, device=DEV).bfloat16() for y in x)
    cache = torch.full((3, H, 1, 32 * D + 16), 0x7f, dtype=torch.uint8, device=DEV)
    raw = cache.cpu().numpy()
    slots = [16 + i for i in range(16)] + list(range(16)) + [20, 19, 23, 21, 16, 17, 33, 34]
    at = 0
    for n in [1] * 9 + [3, 4, 5, 6, 4, 1, 2, 3, 2]:
        pick = slice(at, at + n)
        p8.store(raw, slots[pick], k[pick].double().cpu().numpy(), v[pick].double().cpu().numpy())
        kda.byte_cache_append(k[pick], v[pick], torch.tensor(slots[pick], device=DEV), cache)
        got = cache.cpu().numpy()
        assert np.array_equal(got[..., 32 * D:], raw[..., 32 * D:]), at
        assert np.array_equal(p8.value(got[..., :32 * D]), p8.value(raw[..., :32 * D]),
                              equal_nan=True), at
        at += n


@pytest.mark.parametrize("dtype", DTYPES)
def test_append_non_finite(dtype):
    D = 64
    k = torch.ones((2, 1, D), dtype=dtype, device=DEV)
    v = torch.ones_like(k)
    k[0, 0, 3], k[0, 0, 20], v[1, 0, 40] = float("nan"), float("inf"), float("-inf")
    cache = kda.byte_cache_empty(1, 16, 1, D, DEV)
    slots = torch.arange(2, device=DEV)
    kda.byte_cache_append(k, v, slots, cache)
    assert kda.get_device_error() == 5
    kr, vr = (x.float().cpu().numpy() for x in kda.byte_cache_read(slots, cache, dtype))
    most = 448 * 2.0 ** p8.exponent(1.0)
    assert kr[0, 0, 3] == 0 and kr[0, 0, 20] == most and vr[1, 0, 40] == -most
    kr[0, 0, 3] = kr[0, 0, 20] = vr[1, 0, 40] = 1
    assert (kr == 1).all() and (vr == 1).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_largest_and_smallest_values(dtype):
    most = float(torch.finfo(dtype).max)
    x = torch.tensor([most, -most / 3, 1e-30, 2.0 ** -105, 2.0 ** -110, 1e-45, 0.0], device=DEV,
                     dtype=torch.float64).to(dtype)
    for i in range(len(x)):
        k = x[i:].repeat(64)[:64].reshape(1, 1, 64)
        cache, raw = kda.byte_cache_empty(1, 16, 1, 64, DEV), np.zeros((1, 1, 1, 2064), np.uint8)
        slots = torch.zeros(1, dtype=torch.int64, device=DEV)
        kda.byte_cache_append(k, -k, slots, cache)
        p8.store(raw, [0], k.double().cpu().numpy(), -k.double().cpu().numpy())
        kr, vr = kda.byte_cache_read(slots, cache, dtype)
        assert np.array_equal(kr.double().cpu().numpy(), p8.load(raw, [0])[0])
        assert torch.equal(vr, -kr)


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_value_of_16_bits(dtype):
    """Every finite bf16 number, alone in its block and beside one that sets the exponent."""
    bits = torch.arange(1 << 16, device=DEV).to(torch.int16)
    x = bits.view(torch.bfloat16)
    x = x[x.isfinite()].to(dtype)
    x = torch.cat([x, x.new_zeros(-len(x) % 64)])
    T = len(x) // 64
    k = x.reshape(T, 1, 64)
    v = k[:, :, 63:].expand(T, 1, 64).contiguous()
    cache = kda.byte_cache_empty(T, 16, 1, 64, DEV)
    raw = np.zeros((T, 1, 1, 2064), np.uint8)
    slots = torch.arange(T, device=DEV) * 16
    kda.byte_cache_append(k, v, slots, cache)
    p8.store(raw, slots.tolist(), k.double().cpu().numpy(), v.double().cpu().numpy())
    for a, b in zip(p8.load(raw, slots.tolist()), kda.byte_cache_read(slots, cache, dtype)):
        assert np.array_equal(b.double().cpu().numpy(), a)


def test_bad_slots_are_skipped():
    cache = torch.full((2, 1, 1, 32 * 64 + 16), 7, dtype=torch.uint8, device=DEV)
    x = torch.randn((3, 1, 64), device=DEV)
    for bad in (32, -2, 1 << 40):
        slots = torch.tensor([bad, -1, bad], device=DEV)
        kda.byte_cache_append(x, x, slots, cache)
        assert kda.get_device_error() == 5
        assert (cache == 7).all()
        k, v = kda.byte_cache_read(slots, cache, torch.float32)
        assert kda.get_device_error() == 5
        assert not k.any() and not v.any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,strides", [(1, 3, (0, 160)), (1, 3, (1 << 40, 160)),
                                         (5, 1, (200, 0)), (5, 1, (200, 1 << 40))])
def test_append_strides_of_single_tokens_and_heads_say_nothing(dtype, T, H, strides):
    x = torch.randn((2, T, H, 128), device=DEV).to(dtype)
    room = torch.full((2, 2000), 9.0, dtype=dtype, device=DEV)
    k, v = (room[i].as_strided((T, H, 128), strides + (1,)) for i in range(2))
    k.copy_(x[0]), v.copy_(x[1])
    slots = torch.arange(3, 3 + T, device=DEV)
    caches = [torch.full((1, H, 1, 32 * 128 + 16), 120, dtype=torch.uint8, device=DEV)
              for _ in range(2)]
    kda.byte_cache_append(x[0], x[1], slots, caches[0])
    kda.byte_cache_append(k, v, slots, caches[1])
    assert torch.equal(*caches)


def test_append_takes_broadcast_rows():
    x = torch.randn((2, 1, 2, 64), device=DEV)
    slots = torch.arange(20, device=DEV)
    caches = [torch.zeros((2, 2, 1, 32 * 64 + 16), dtype=torch.uint8, device=DEV)
              for _ in range(2)]
    wide = x.expand(2, 20, 2, 64)
    kda.byte_cache_append(wide[0], wide[1], slots, caches[0])
    kda.byte_cache_append(wide[0].contiguous(), wide[1].contiguous(), slots, caches[1])
    assert torch.equal(*caches)


# --------------------------------------------------------------- attention ---

class Problem:
    """Requests over a cache of random pages; the bytes no request holds are random too, codes
    of NaN among them.  ``spread``: range of the blocks' powers of two."""

    def __init__(self, kv, new, Hq, Hk, D, P, dtype, seed=0, extra_pages=2, qscale=1.5, spread=2,
                 k_spread=0):
        rng = np.random.RandomState(seed)
        self.kv, self.new, self.Hq, self.Hk, self.D, self.P = kv, new, Hq, Hk, D, P
        need = [-(-n // P) for n in kv]
        pages = sum(need) + extra_pages
        ids = rng.permutation(pages)
        self.table = np.full((len(kv), max(need + [1])), -7)
        raw = rng.randint(0, 256, (pages, Hk, P // 16, 32 * D + 16)).astype(np.uint8)
        raw[..., :32 * D][rng.rand(*raw.shape[:3], 32 * D) < 0.2] = 0x7f
        self.ks, self.vs, self.ve = [], [], []
        at = 0
        for b, n in enumerate(kv):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            k = rng.randn(n, Hk, D) * np.exp2(rng.randint(-2, 2, (Hk, D)))
            if k_spread:
                k *= np.repeat(np.exp2(rng.randint(-k_spread, 1, (n // 16 + 1, Hk, 1))), 16, 0)[:n]
            v = rng.randn(n, Hk, D)
            v *= np.repeat(np.exp2(rng.randint(-spread, spread + 1, (n // 16 + 1, Hk, 1))), 16, 0)[:n]
            if n:
                pos = np.arange(n)
                slots = self.table[b, pos // P] * P + pos % P
                p8.store(raw, slots, k, v)
                k, v = p8.load(raw, slots)
                self.ve.append(raw[self.table[b, pos // P], :, pos % P // 16, 32 * D + 1].astype(float))
            else:
                self.ve.append(np.zeros((0, Hk)))
            self.ks.append(k)
            self.vs.append(v)
        self.cache = torch.tensor(raw, device=DEV)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(int)
        self.q = torch.tensor(rng.randn(self.cu[-1], Hq, D) * qscale, device=DEV).to(dtype)

    def call(self, **kw):
        q = kw.pop("q", self.q)
        kw.setdefault("max_new", max(self.new + [1]))
        return kda.byte_cache_attention(q, kw.pop("cache", self.cache), i32(kw.pop("table", self.table)),
                                    i32(kw.pop("kv", self.kv)), i32(kw.pop("cu", self.cu)),
                                    return_lse=True, **kw)

    def check(self, out, lse, scale=None, only=None):
        scale = self.D ** -0.5 if scale is None else scale
        q = self.q.double().cpu().numpy()
        out_h, lse_h = out.double().cpu().numpy(), lse.double().cpu().numpy()
        bf16 = self.q.dtype == torch.bfloat16
        for b, (L, n) in enumerate(zip(self.kv, self.new)):
            if only is not None and b not in only:
                continue
            rows = slice(self.cu[b], self.cu[b + 1])
            o, z, mass, _, size = pc.attention(q[rows], self.ks[b], self.vs[b], scale)
            under = np.exp2(self.ve[b].max(0, initial=0) - self.ve[b])[..., None]
            flat = pc.attention(q[rows], self.ks[b], self.vs[b] * under, scale)[3]
            tol = (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(o) + mass * (
                (2.0 ** -11 if bf16 else 2.0 ** -21) + size[..., None] * 2.0 ** -16 +
                (L + 64) * 2.0 ** -23) + flat * 2.0 ** -31
            err = np.abs(out_h[rows] - o)
            assert np.isfinite(out_h[rows]).all(), f"request {b}"
            assert not (err > tol).any(), (b, L, n, float((err / np.maximum(tol, 1e-300)).max()))
            empty = np.isinf(z)
            assert np.array_equal(np.isinf(lse_h[rows]), empty) and (lse_h[rows][empty] < 0).all()
            ltol = size * 2.0 ** -16 + (L + 64) * 2.0 ** -23 + np.abs(np.where(empty, 0, z)) * 2.0 ** -22
            assert (np.abs(np.where(empty, 0, lse_h[rows] - np.where(empty, 0, z))) <= ltol).all(), b


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
@pytest.mark.parametrize("new", [1, 3, 60])
@pytest.mark.parametrize("spread", [9, 30])
def test_values_of_unequal_size(dtype, new, spread):
    """Blocks of V whose powers of two lie far apart, rising and falling along a request."""
    p = Problem([500, 77, 130], [new, new, 1], 4, 2, 128, 32, dtype, seed=new, spread=spread)
    p.check(*p.call())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 3, 60])
@pytest.mark.parametrize("spread", [6, 40])
def test_keys_of_unequal_size(dtype, new, spread):
    """The same of K: scores of most blocks are small beside those of a few."""
    p = Problem([500, 77, 130], [new, new, 1], 4, 2, 128, 32, dtype, seed=new, k_spread=spread)
    p.check(*p.call())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 60])
def test_a_large_weight_on_small_values(dtype, new):
    """The row's largest weight falls on a block of tiny values, as on a sequence's first token:
    the output is the other blocks', with weights of 2^-9 to 2^-14 of the largest."""
    p = Problem([200], [new], 2, 1, 64, 32, dtype, seed=5, spread=0)
    raw = p.cache.cpu().numpy()
    pos = np.arange(200)
    slots = p.table[0, pos // 32] * 32 + pos % 32
    k, v = p.ks[0].copy(), p.vs[0].copy()
    k[:] = 0.01 * k
    k[0] = 1.0
    v[:16] *= 2.0 ** -20
    p8.store(raw, slots, k, v)
    p.ks[0], p.vs[0] = p8.load(raw, slots)
    p.ve[0] = raw[p.table[0, pos // 32], :, pos % 32 // 16, 32 * 64 + 1].astype(float)
    p.cache = torch.tensor(raw, device=DEV)
    p.q = torch.ones_like(p.q)
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
    odd = torch.full((T, 4, 131), 9.0, dtype=dtype, device=DEV)
    odd[..., 1:129] = p.q
    for q in (wide[:, 1], odd[..., 1:129]):
        for a, b in zip(base, p.call(q=q)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("new", [1, 40])
def test_scales_and_large_scores(new):
    p = Problem([150, 77], [new, new], 4, 2, 64, 32, torch.bfloat16, seed=9, qscale=200.0)
    p.check(*p.call(scale=1.0), scale=1.0)
    for scale in (0.0, -0.2, 0.07):
        for dtype in DTYPES:
            p = Problem([150, 77], [new, new], 4, 2, 64, 32, dtype, seed=9)
            p.check(*p.call(scale=scale), scale=np.float64(np.float32(scale)))


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
        for x in (hidden.ks, hidden.vs, hidden.ve):
            x[1] = x[1][keep]
        hidden.kv = [100, 68, 100]
        if new == 1:  # (rows inside the hidden page see less than this makes of them)
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


def test_empty_rows_and_empty_batch():
    p = Problem([0, 0], [1, 4], 4, 2, 64, 16, torch.float32)
    p.check(*p.call())
    p = Problem([9, 0], [0, 0], 4, 2, 64, 16, torch.float32)
    out, lse = p.call()
    assert out.shape == (0, 4, 64)


def test_pages_beyond_32_bits():
    """A cache of more than 2^32 bytes, the request's pages at its end."""
    Hk, D, P = 8, 128, 256
    group = 32 * D + 16
    pages = (1 << 32) // (Hk * P // 16 * group) + 40
    small = Problem([700], [1], 8, Hk, D, P, torch.bfloat16, seed=1, extra_pages=0)
    cache = torch.empty((pages, Hk, P // 16, group), dtype=torch.uint8, device=DEV)
    n = small.cache.shape[0]
    cache[-n:] = small.cache
    table = np.where(small.table >= 0, small.table + pages - n, -1)
    small.check(*small.call(cache=cache, table=table))
    slots = torch.tensor([(pages - 1) * P, (pages - 40) * P], device=DEV)
    x = torch.randn((2, Hk, D), device=DEV)
    kda.byte_cache_append(x, -x, slots, cache)
    k, v = kda.byte_cache_read(slots, cache, torch.float32)
    assert torch.equal(k, -v) and (k - x).abs().max() <= x.abs().max() / 16
    # the last page copied to the first and back
    last = cache[-1].clone()
    kda.cache_copy(cache, i32([[pages - 1, 0, P]]))
    cache[-1].zero_()
    kda.cache_copy([cache], i32([[0, pages - 1, P - 15]]))
    assert torch.equal(cache[-1], last) and torch.equal(cache[0], last)


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
        kda.byte_cache_attention(p.q, p.cache, table, kv, cu, max_new=new, out=out)
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


@pytest.mark.parametrize("new", [1, 60])
def test_callers_workspace(new):
    p = Problem([90, 300], [new, new], 8, 2, 128, 32, torch.bfloat16, seed=7)
    base = p.call()
    size = kda.byte_cache_attention_workspace_size(p.cache, 2, 2 * new, 8, new, p.table.shape[1],
                                               torch.bfloat16)
    room = torch.full((size + 512,), 0xff, dtype=torch.uint8, device=DEV)
    off = -room.data_ptr() % 256
    for a, b in zip(base, p.call(workspace=room[off:off + size])):
        assert torch.equal(a, b)
    assert (room[off + size:] == 0xff).all() and (room[:off] == 0xff).all()
    with pytest.raises(kda.KDAError):
        p.call(workspace=room[off:off + size - 1])
    with pytest.raises(kda.KDAError):
        p.call(workspace=room[off + 16:off + 16 + size])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kv,new", [([70, 2000, 33], [1, 1, 1]), ([70, 2000, 33], [3, 5, 0]),
                                    ([70, 900], [60, 200])])
def test_expired_wait_reports_timeout_and_recovers(dtype, kv, new):
    p = Problem(kv, new, 8, 2, 128, 32, dtype, seed=12)
    base = p.call()
    kda.testing_inject_wait_timeout()
    p.call()
    assert kda.get_device_error() == 4
    for a, b in zip(base, p.call()):
        assert torch.equal(a, b)


def test_calls_on_two_streams_at_once():
    """Append, attention and read of two caches on a stream each, workspaces of their own."""
    ps = [Problem([700, 90], [n, n], 8, 2, 128, 32, torch.bfloat16, seed=n) for n in (1, 60)]
    base = [p.call() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (p, st) in enumerate(zip(ps, streams)):
            with torch.cuda.stream(st):
                got[i].append(p.call())
    torch.cuda.synchronize()
    for b, gs in zip(base, got):
        for g in gs:
            assert all(torch.equal(x, y) for x, y in zip(b, g))


def test_graphs_that_share_a_workspace():
    """Two captured calls, of another shape each, with one workspace, replayed in turn."""
    ps = [Problem([700, 90], [n, n], 8, 2, 128, 32, torch.bfloat16, seed=n) for n in (1, 60)]
    base = [p.call() for p in ps]
    size = max(kda.byte_cache_attention_workspace_size(
        p.cache, 2, p.q.shape[0], 8, max(p.new), p.table.shape[1], torch.bfloat16) for p in ps)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for p in ps:
        args = [i32(x) for x in (p.table, p.kv, p.cu)]
        g = torch.cuda.CUDAGraph()
        out = torch.zeros_like(p.q)
        with torch.cuda.graph(g):
            kda.byte_cache_attention(p.q, p.cache, *args, max_new=max(p.new), out=out, workspace=ws)
        graphs.append((g, args))
        outs.append(out)
    for _ in range(3):
        for (g, _), out, b in zip(graphs, outs, base):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, b[0])


@pytest.mark.parametrize("D,new", [(64, 1), (128, 1), (128, 3)])
def test_fp32_sums_of_a_long_row(D, new):
    """fp32 outputs over 9001 keys: errors of sums that the tensor cores truncate would show."""
    p = Problem([9001], [new], 4, 2, D, 64, torch.float32, seed=2, qscale=0.3, spread=0)
    out, lse = p.call()
    q = p.q.double().cpu().numpy()
    o = pc.attention(q, p.ks[0], p.vs[0], D ** -0.5)[0]
    err = np.linalg.norm(out.double().cpu().numpy() - o) / np.linalg.norm(o)
    # weights 2^-22, scores of 1 off by 2^-21 each at random, sums over 9001 in pieces: 2^-23
    # sqrt(9001 / 16)
    assert err <= 3e-6, err


def test_append_then_attend():
    """The step a server makes: tables, append, attention, over several steps, windows that were
    rejected among them."""
    P, B, Hk, Hq, D = 16, 3, 2, 8, 64
    rng = np.random.RandomState(3)
    cache = torch.full((30, Hk, 1, 32 * D + 16), 0x7f, dtype=torch.uint8, device=DEV)
    raw = cache.cpu().numpy()
    table = torch.full((B, 6), -1, dtype=torch.int32, device=DEV)
    ring = torch.arange(30, dtype=torch.int32, device=DEV)
    span = torch.tensor([0, 30], device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    p = Problem([], [], Hq, Hk, D, P, torch.bfloat16)
    for new, back in (([20, 33, 5], 0), ([1, 1, 1], 0), ([3, 0, 2], 0), ([4, 4, 4], 0),
                      ([2, 1, 3], 3), ([1, 1, 1], 0)):
        T = sum(new)
        k, v = (torch.tensor(rng.randn(T, Hk, D) * np.exp2(rng.randint(-3, 4, (T, 1, 1))),
                             device=DEV).bfloat16() for _ in range(2))
        p.q = torch.tensor(rng.randn(T, Hq, D), device=DEV).bfloat16()
        lens, cu, slots, span = kda.cache_tables(lens, lens - back, i32(new), table, ring, span,
                                                 page_size=P, max_tokens=T)
        kda.byte_cache_append(k, v, slots, cache)
        p8.store(raw, slots.tolist(), k.double().cpu().numpy(), v.double().cpu().numpy())
        out, lse = kda.byte_cache_attention(p.q, cache, table, lens, cu, max_new=max(new),
                                        return_lse=True)
        p.cu = np.concatenate([[0], np.cumsum(new)]).astype(int)
        p.new, p.kv = new, lens.tolist()
        t = table.cpu().numpy()
        p.ks, p.vs, p.ve = [], [], []
        for b in range(B):
            pos = np.arange(p.kv[b])
            held = p8.load(raw, t[b, pos // P] * P + pos % P)
            p.ks.append(held[0])
            p.vs.append(held[1])
            p.ve.append(raw[t[b, pos // P], :, pos % P // 16, 32 * D + 1].astype(float))
        p.check(out, lse)
