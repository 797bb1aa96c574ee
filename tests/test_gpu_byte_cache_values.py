"""GPU tests of the 8-bit cache's attention where its powers of two and fp32's steps bind: the
largest block is one that earlier rows do not see, scores of tens of millions."""
import numpy as np
import pytest
import torch

import linear_attention_layer_gb300 as kda
from oracle import byte_cache as p8
from oracle import paged_cache as pc
from tests.test_gpu_byte_cache import Problem
from tests.test_gpu_cache import DEV, DTYPES, _device  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,kv", [(3, 97), (9, 337), (40, 321), (70, 1057)])
@pytest.mark.parametrize("up_k,up_v", [(0, 12), (0, 20), (8, 8), (12, 0)])
def test_the_largest_block_is_one_that_earlier_rows_do_not_see(dtype, new, kv, up_k, up_v):
    """The newest token begins a block whose values (keys) lie 2^up above all others.  A row that
    does not see it may share a tile, and with it the unit 2^E of its weights or halves, with one
    that does.  Beside the terms of tests/test_gpu_byte_cache.py, for each row:
      - on the kernel for few rows (fp32, or up to 48 rows a kv head), weights off by 2^-32 of the
        row's largest under E: |v_j| 2^(E - e_j) 2^-32 of the sum of weights each;
      - in chunks, values off by half a step of a half's smallest numbers, 2^(E - 25), and scores by
        sum_c |q_c| 2^(E_k - 25) each, whose weights e^that."""
    p = Problem([kv, 40], [new, 1], 4, 2, 64, 32, dtype, seed=new, qscale=0.5, spread=1)
    raw, pos = p.cache.cpu().numpy(), np.arange(kv)
    slots = p.table[0, pos // 32] * 32 + pos % 32
    k, v = p.ks[0].copy(), p.vs[0].copy()
    assert kv % 16 == 1
    k[-1] *= 2.0 ** up_k / 2
    v[-1] *= 2.0 ** up_v
    p8.store(raw, slots, k, v)
    k, v = p8.load(raw, slots)
    ek, ev = (raw[p.table[0, pos // 32], :, pos % 32 // 16, 32 * 64 + i].astype(float) - 127
              for i in range(2))
    p.cache = torch.tensor(raw, device=DEV)
    out, lse = p.call()
    q, out_h, lse_h = (x.double().cpu().numpy()[:new] for x in (p.q, out, lse))
    bf16, scale = dtype == torch.bfloat16, 64 ** -0.5
    chunk = bf16 and new * 2 > 48
    o, z, mass, flat, size = pc.attention(q, k, v, scale)
    top_v, top_k = ev.max(0).repeat(2), ek.max(0).repeat(2)  # of the query heads
    if chunk:
        lost = 2.0 ** (top_v - 25)[None, :, None]
        score = np.abs(q).sum(-1) * scale * 2.0 ** (top_k - 25)
    else:
        under = np.exp2(ev.max(0) - ev)[..., None]
        lost = pc.attention(q, k, v * under, scale)[3] * 2.0 ** -32
        score = np.zeros(q.shape[:2])
    size = size * 2.0 ** -17 + score  # what a score is off by
    step = 2.0 ** -8 if bf16 else 2.0 ** -24
    tol = step * np.abs(o) + lost + flat * 2.0 ** -32 + mass * (
        (2.0 ** -11 if bf16 else 2.0 ** -21) + 2 * size[..., None] + (kv + 64) * 2.0 ** -23)
    err = np.abs(out_h - o)
    assert (err <= tol).all(), float((err / tol).max())
    assert (np.abs(lse_h - z) <= 2 * size + (kv + 64) * 2.0 ** -23 + np.abs(z) * 2.0 ** -22).all()
    p.kv, p.new, p.cu, p.q = p.kv[1:], p.new[1:], p.cu[1:] - new, p.q[new:]
    p.ks, p.vs, p.ve = p.ks[1:], p.vs[1:], p.ve[1:]
    p.check(out[new:], lse[new:])  # the other request is none of this


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [1, 4, 60])
def test_scores_of_tens_of_millions(dtype, new):
    """Two keys whose scores lie 12 (in powers of two) apart at 5.0e7 of those, where fp32 steps by
    4, in different tiles of every request: the reference and what passes it are rounded to
    that, and weights have to fit a half all the same.  The scores' common factor is off by 2^-23,
    their difference with it."""
    B, Hk, G, D, P, L, scale = 1000 if new < 60 else 64, 4, 2, 64, 64, 192, 22711.783203125
    k, v = np.zeros((L, Hk, D)), np.zeros((L, Hk, D))
    k[3, :, 0], k[100, :, 0] = 1536.0, 1536.0
    k[100, :, 16] = 3.0
    v[3], v[100], v[50] = 6.0, 3.0, -6.0
    v[100, :, ::16] = 6.0
    raw = np.zeros((3, Hk, P // 16, 32 * D + 16), np.uint8)
    p8.store(raw, np.arange(L), k, v)
    held = p8.load(raw, np.arange(L))
    assert np.array_equal(held[0], k) and np.array_equal(held[1], v)
    q = torch.zeros((B * new, G * Hk, D), dtype=dtype, device=DEV)
    q[..., 0], q[..., 16] = 1.0, 2.0 ** -13
    ints = dict(dtype=torch.int32, device=DEV)
    out = kda.byte_cache_attention(
        q, torch.tensor(raw, device=DEV), torch.tensor([[0, 1, 2]] * B, **ints),
        torch.full((B,), L, **ints), torch.arange(0, (B + 1) * new, new, **ints), max_new=new,
        scale=scale)
    p = np.exp(-scale * 3 * 2.0 ** -13)
    want = (p * v[3, 0] + v[100, 0]) / (1 + p)
    step = 2.0 ** -8 + 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -24 + 2.0 ** -21
    tol = want * (step + 12 * 2.0 ** -23)
    worst = float((np.abs(out.double().cpu().numpy() - want) / tol).max())
    assert worst <= 1, worst


@pytest.mark.parametrize("dtype", DTYPES)
def test_an_exponent_stays_until_the_block_is_begun_anew(dtype):
    """In zeroed bytes from any place on; what a rejected draft has raised stays for the tokens that
    follow, and falls with the next token at the first place."""
    cache = torch.zeros((1, 1, 1, 32 * 64 + 16), dtype=torch.uint8, device=DEV)
    small = 2.0 ** -12

    def append(place, value):
        x = torch.full((1, 1, 64), value, device=DEV).to(dtype)
        kda.byte_cache_append(x, -x, torch.tensor([place], device=DEV), cache)

    def held(place):
        k, v = kda.byte_cache_read(torch.tensor([place], device=DEV), cache, dtype)
        assert torch.equal(k, -v) and (k == k[0, 0, 0]).all()
        return float(k[0, 0, 0]), int(cache[0, 0, 0, 32 * 64]) - 127

    append(3, small)
    assert held(3) == (small, -20)  # 2^-12 <= 448 2^-20
    append(4, 1.0)
    assert held(4) == (1.0, -8) and held(3)[0] == small
    append(5, 64.0)  # a draft
    assert held(5) == (64.0, -2) and held(3)[0] == 0.0  # 2^-10 of the unit, half of a step: to even
    append(5, small)
    assert held(5) == (0.0, -2) and held(4)[0] == 1.0
    append(0, small)
    assert held(0) == (small, -20)
