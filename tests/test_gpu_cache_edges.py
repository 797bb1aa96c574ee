"""GPU tests of the 4-bit paged cache where a call is easily answered wrongly: unusual strides,
long fp32 rows, weights far below the largest, hidden pages, waits that run out."""
import numpy as np
import pytest
import torch

import linear_attention_layer_gb300 as kda
from oracle import paged_cache as pc
from tests.test_gpu_cache import DEV, DTYPES, Problem, _device  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- strides ---

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,strides", [(1, 4, (0, 160)), (1, 4, (1 << 40, 160)),
                                         (6, 1, (200, 0)), (6, 1, (200, 1 << 40))])
def test_strides_of_single_tokens_and_heads_say_nothing(dtype, T, H, strides):
    """torch leaves any stride in a dimension of one element."""
    p = Problem([50], [T], H, 1, 128, 16, dtype, seed=T)
    base = p.call()
    room = torch.full((2000,), 9.0, dtype=dtype, device=DEV)
    q = room.as_strided((T, H, 128), strides + (1,))
    q.copy_(p.q)
    assert q.stride()[:2] == strides and not q.is_contiguous()
    for a, b in zip(base, p.call(q=q)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,strides", [(1, 3, (0, 160)), (1, 3, (1 << 40, 160)),
                                         (5, 1, (200, 0)), (5, 1, (200, 1 << 40))])
def test_append_strides_of_single_tokens_and_heads_say_nothing(dtype, T, H, strides):
    x = torch.randn((2, T, H, 128), device=DEV).to(dtype)
    room = torch.full((2, 2000), 9.0, dtype=dtype, device=DEV)
    k, v = (room[i].as_strided((T, H, 128), strides + (1,)) for i in range(2))
    k.copy_(x[0]), v.copy_(x[1])
    slots = torch.arange(3, 3 + T, device=DEV)
    caches = [torch.zeros((1, H, 1, 18 * 128), dtype=torch.uint8, device=DEV) for _ in range(2)]
    kda.cache_append(x[0], x[1], slots, caches[0])
    kda.cache_append(k, v, slots, caches[1])
    assert torch.equal(*caches)


def test_append_takes_broadcast_rows():
    """One key and value for every token: stride 0 is what it says."""
    x = torch.randn((2, 1, 2, 64), device=DEV)
    slots = torch.arange(20, device=DEV)
    caches = [torch.zeros((2, 2, 1, 18 * 64), dtype=torch.uint8, device=DEV) for _ in range(2)]
    wide = x.expand(2, 20, 2, 64)
    kda.cache_append(wide[0], wide[1], slots, caches[0])
    kda.cache_append(wide[0].contiguous(), wide[1].contiguous(), slots, caches[1])
    assert torch.equal(*caches)


# ------------------------------------------------- waits that run out ---

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kv,new", [([70, 2000, 33], [1, 1, 1]), ([70, 2000, 33], [3, 5, 0]),
                                    ([700, 333, 90], [200, 1, 40])])
def test_expired_wait_reports_timeout_and_recovers(dtype, kv, new):
    """An input wait made to run out by the testing hook, in a decode step, windows and (bf16)
    the chunk kernel: the calls end with KDA_ERR_TIMEOUT in the error word, and the next one on
    the same context is right."""
    p = Problem(kv, new, 8, 2, 128, 32, dtype, seed=21)
    base = p.call()
    kda.testing_inject_wait_timeout(1)
    p.call()
    assert kda.get_device_error() == 4
    again = p.call()
    assert kda.get_device_error() == 0
    for a, b in zip(base, again):
        assert torch.equal(a, b)
    p.check(*again)


# ------------------------------------------------------ 31-bit borders ---

def test_tables_with_room_for_the_most_tokens():
    """max_tokens = 2^31 - 1: counters that step past it do not wrap."""
    P, most = 64, 2 ** 31 - 1
    table = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    ring = torch.tensor([4, 2, 0, 1, 3], dtype=torch.int32, device=DEV)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    kv, cu, slots, span = kda.cache_tables(
        zero, zero, torch.tensor([70, 9], dtype=torch.int32, device=DEV), table, ring,
        torch.tensor([0, 5], device=DEV), page_size=P, max_tokens=most)
    assert kv.tolist() == [70, 9] and cu.tolist() == [0, 70, 79] and span.tolist() == [3, 5]
    want = list(range(4 * P, 5 * P)) + list(range(2 * P, 2 * P + 6)) + list(range(9))
    assert slots.numel() == most and slots[:79].tolist() == want
    for part in slots[79:].split(1 << 28):
        assert bool((part == -1).all())


@pytest.mark.parametrize("new", [1, 60])
def test_lengths_that_round_up_past_31_bits_are_refused(new):
    """A table of one page over and over may claim them; such a request is skipped."""
    p = Problem([100], [new], 4, 2, 64, 32, torch.bfloat16)
    cache = torch.zeros((1, 2, 256, 18 * 64), dtype=torch.uint8, device=DEV)
    table = torch.zeros((1, 1 << 19), dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, new], dtype=torch.int32, device=DEV)
    for kv in (2 ** 31 - 1, 2 ** 31 - 127):
        out = torch.full_like(p.q, 3.0)
        kda.cache_attention(p.q, cache, table, torch.tensor([kv], dtype=torch.int32, device=DEV),
                            cu, max_new=new, out=out)
        assert kda.get_device_error() == 5
        assert bool((out == 3.0).all())


# ------------------------------------------------------- fp32 outputs ---

@pytest.mark.parametrize("D,new", [(64, 1), (128, 1), (64, 5), (128, 5)])
def test_fp32_keeps_weights_far_below_the_largest(D, new):
    """40000 keys of weight e^-23 = 2^-33.2 behind a dominant one whose values are zero in half of
    the channels.  A weight is held in two halves, the second 2^11 times larger: 2^-11 of it, or
    2^-36 where the row's largest has 2^7 at least, 2^-43 of it."""
    L, Hq = 40000, 4
    p = Problem([L], [new], Hq, 1, D, 64, torch.float32, seed=D)
    k, v = np.zeros((L, 1, D)), np.ones((L, 1, D))
    k[777, 0, 0] = 6.0  # an exact code
    v[777, 0, : D // 2] = 0.0
    raw = p.cache.cpu().numpy()
    pos = np.arange(L)
    pc.store(raw, p.table[0, pos // 64] * 64 + pos % 64, k, v)
    p.cache = torch.tensor(raw, device=DEV)
    v = pc.dequantise(*pc.quantise(v))
    q = np.zeros((new, Hq, D))
    q[..., 0] = 23.0 / 6.0 * D ** 0.5
    p.q = torch.tensor(q, device=DEV).float()
    out, lse = p.call()
    want, z, mass, flat, size = pc.attention(p.q.double().cpu().numpy(), k, v, D ** -0.5)
    assert (want[..., 0] > 4e-6).all() and (want[..., -1] > 0.9).all()
    tol = 2.0 ** -24 * want + mass * (2.0 ** -21 + size[..., None] * 2.0 ** -16) + flat * 2.0 ** -43
    worst = float((np.abs(out.double().cpu().numpy() - want) / tol).max())
    assert worst <= 1, worst


@pytest.mark.parametrize("D,new,Hq,Hk", [(128, 1, 4, 2), (64, 1, 6, 3), (128, 6, 4, 2), (64, 3, 8, 2)])
def test_fp32_sums_of_a_long_row(D, new, Hq, Hk):
    """The error of a request's outputs over 9001 keys, by its norm, in a batch of 1000 (of one
    request's tokens and queries over and over), where a warp adds up whole rows.  Weights are
    off by 2^-22 (two halves) and by their score's error, about 2^-24 of the magnitudes that it
    adds up (its sums are rounded every 32 products): independent of the values' signs, so the
    outputs are off by no more than that.  Sums left to the tensor cores, which cut off, or
    queries or weights in one half are off by more."""
    B = 1000
    p = Problem([9001], [new], Hq, Hk, D, 64, torch.float32, seed=D + new)
    want, z, mass, flat, size = pc.attention(p.q.double().cpu().numpy(), p.ks[0], p.vs[0], D ** -0.5)
    ints = dict(dtype=torch.int32, device=DEV)
    out = kda.cache_attention(p.q.repeat(B, 1, 1), p.cache,
                              torch.tensor(p.table, **ints).repeat(B, 1),
                              torch.full((B,), 9001, **ints),
                              torch.arange(0, (B + 1) * new, new, **ints), max_new=new)
    err = (out.double() - torch.tensor(want, device=DEV).repeat(B, 1, 1)).reshape(B, -1).norm(dim=1)
    worst = float(err.max()) / np.linalg.norm(want)
    assert worst <= 2.0 ** -22 + size.mean() * 2.0 ** -24, worst


# ------------------------------------------------------- large scores ---

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 4, 60])
def test_scores_of_tens_of_millions(dtype, new):
    """Two keys whose scores lie 12 (in powers of two) apart at 3.4e7, where fp32 steps by 2 to
    4, in different tiles of every request: beside a reference of this size the limit up to
    which weights fit a half has to be rounded down.  The scores' common factor is off by 2^-23,
    their difference with it."""
    B, Hk, G, D, P, L, scale = 1000 if new < 60 else 64, 4, 2, 64, 64, 192, 22711.783203125
    k, v = np.zeros((L, Hk, D)), np.zeros((L, Hk, D))
    k[3, :, 0], k[100, :, 0] = 1536.0, 1536.0
    k[100, :, 16], k[100, :, 17] = 3.0, 6.0  # the latter for the block's scale
    v[3], v[100], v[50] = 6.0, 3.0, -6.0
    v[100, :, ::16] = 6.0
    raw = np.zeros((3, Hk, P // 16, 18 * D), np.uint8)
    pos = np.arange(L)
    pc.store(raw, pos, k, v)
    q = torch.zeros((B * new, G * Hk, D), dtype=dtype, device=DEV)
    q[..., 0], q[..., 16] = 1.0, 2.0 ** -13
    ints = dict(dtype=torch.int32, device=DEV)
    out = kda.cache_attention(
        q, torch.tensor(raw, device=DEV), torch.tensor([[0, 1, 2]] * B, **ints),
        torch.full((B,), L, **ints), torch.arange(0, (B + 1) * new, new, **ints), max_new=new,
        scale=scale)
    p = np.exp(-scale * 3 * 2.0 ** -13)
    want = (p * v[3, 0] + v[100, 0]) / (1 + p)
    step = 2.0 ** -8 + 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -24 + 2.0 ** -21
    tol = want * (step + 12 * 2.0 ** -23)
    worst = float((np.abs(out.double().cpu().numpy() - want) / tol).max())
    assert worst <= 1, worst


# ------------------------------------------------- pages, workspaces, many ---

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 5, 40])
@pytest.mark.parametrize("page", [-1, 1 << 20])
def test_rows_see_what_a_hidden_page_leaves(dtype, new, page):
    """Values, row by row, of a request one page of which is not in the cache: a row sees the
    tokens up to its own but for that page's."""
    p = Problem([100, 90], [new, 1], 8, 2, 128, 32, dtype, seed=14)
    table = p.table.copy()
    table[0, 2] = page  # tokens 64 .. 95
    out, lse = p.call(table=table)
    assert kda.get_device_error() == 5
    p.check(out, lse, only={1})
    rows = Problem([1] * new, [1] * new, 8, 2, 128, 32, dtype)  # its check, a request a row
    rows.q, ks, vs = p.q[:new], p.ks[0], p.vs[0]
    keep = [np.r_[0:64, 96:100][: sum(t <= 100 - new + i for t in np.r_[0:64, 96:100])]
            for i in range(new)]
    rows.ks, rows.vs = [ks[k] for k in keep], [vs[k] for k in keep]
    rows.kv = [len(k) for k in keep]
    rows.check(out[:new], lse[:new])


@pytest.mark.parametrize("new", [1, 40])
def test_callers_workspace(new):
    p = Problem([300, 70], [new, new], 8, 2, 128, 32, torch.bfloat16, seed=5)
    base = p.call()
    size = kda.cache_attention_workspace_size(p.cache, 2, 2 * new, 8, new, p.table.shape[1],
                                              torch.bfloat16)
    room = torch.full((size + 512,), 255, dtype=torch.uint8, device=DEV)
    for a, b in zip(base, p.call(workspace=room[:size])):
        assert torch.equal(a, b)
    assert bool((room[size:] == 255).all())
    for bad in (room[:size - 1], room[1:size + 1]):  # short; not 256-byte aligned
        with pytest.raises(kda.KDAError):
            p.call(workspace=bad)
    for bad in (room[:size].view(torch.int8), room[::2], "none"):
        with pytest.raises(ValueError):
            p.call(workspace=bad)


def test_many_requests_of_many_rows():
    """More requests, and units of rows, than one pass of the chunk kernel's planner takes."""
    rng = np.random.RandomState(4)
    kv = list(map(int, rng.randint(0, 70, 1100)))
    p = Problem(kv, [9] * len(kv), 32, 1, 64, 16, torch.bfloat16, seed=8)
    p.check(*p.call(), only=set(range(0, 1100, 53)) | {1023, 1024, 1025, 1099})


# -------------------------------------------------------------- rounding ---

@pytest.mark.parametrize("dtype", DTYPES)
def test_every_bf16_value_under_every_scale(dtype):
    """For each E4M3 scale, a block's largest value that gives it and all bf16 values up to that
    one (from 2^-3 of the smallest code's border on; both signs), codes against fp64."""
    bits = np.arange(0x7f80, dtype=np.uint32) << 16
    every = bits.view(np.float32).astype(np.float64)
    scale = pc.nearest(pc.E4M3, every / 6)
    blocks = []
    for sb in range(1, 127):
        tops = every[scale == sb]
        x = every[(every <= tops.max()) & (every >= pc.E4M3[sb] / 32)]
        x = np.pad(x, (0, -len(x) % 14)).reshape(-1, 14)
        top = np.resize(tops, len(x))
        x = np.minimum(x, top[:, None])
        blocks.append(np.concatenate([top[:, None], x, -x[:, :1]], 1))
    blocks = np.concatenate(blocks)
    blocks = np.pad(blocks, ((0, -len(blocks) % 4), (0, 0)))
    blocks[:, 1::2] *= -1
    k = blocks.reshape(-1, 1, 64)
    slots = torch.arange(len(k), device=DEV)
    cache = kda.cache_empty(-(-len(k) // 16), 16, 1, 64, DEV)
    t = torch.tensor(k, device=DEV).to(dtype)
    assert np.array_equal(t.double().cpu().numpy(), k)
    kda.cache_append(t, -t, slots, cache)
    kr, vr = kda.cache_read(slots, cache, dtype)
    want = pc.dequantise(*pc.quantise(k))
    assert np.array_equal(kr.double().cpu().numpy(), want) and torch.equal(kr, -vr)
