"""GPU tests of 8-bit cache appends whose batch comes back to a block: tokens of a block that do not
stand next to one another, up to 16 apart, are left out and reported, as include/kda.h says."""
import numpy as np
import pytest
import torch

import linear_attention_layer_gb300 as kda
from oracle import byte_cache as p8
from tests.test_gpu_cache import DEV, DTYPES, _device  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def _kept(slots):
    """The slots with -1 in place of every run of a block that one of the 16 tokens before it is of."""
    blocks = [s // 16 if s >= 0 else None for s in slots]
    out = list(slots)
    t = 0
    while t < len(slots):
        end = t + 1
        if blocks[t] is not None:
            while end < len(slots) and blocks[end] == blocks[t]:
                end += 1
            if blocks[t] in blocks[max(0, t - 16):t]:
                out[t:end] = [-1] * (end - t)
        t = end
    return out


def _pieces(rng, T, blocks):
    """Slots of T tokens: pieces of up to 17, each with the slots of a few blocks of its own in any
    order, -1 between them."""
    slots, ids = [], list(rng.permutation(blocks))
    while len(slots) < T:
        n, some = int(rng.randint(1, 18)), [int(ids.pop()) for _ in range(rng.randint(1, 4))]
        mine = rng.permutation([b * 16 + i for b in some for i in range(16)])[:n]
        if rng.rand() < 0.5:
            mine = sorted(mine)  # the blocks one after another: nothing to report
        slots += [-1 if rng.rand() < 0.1 else int(s) for s in mine]
    return slots[:T]


def _check(slots, H, D, dtype, P=32, blocks=None, heads=None):
    T = len(slots)
    pages = -(-(blocks or max(slots) // 16 + 1) * 16 // P)
    heads = list(range(H)) if heads is None else heads
    g = torch.Generator(device=DEV).manual_seed(T + D)
    src = torch.randn((T, 2 * H, D), device=DEV, generator=g)
    src *= torch.exp2(torch.randint(-6, 7, (T, 1, 1), device=DEV, generator=g).float())
    src = src.to(dtype)
    cache = torch.randint(0, 120, (pages, H, P // 16, 32 * D + 16), dtype=torch.uint8, device=DEV,
                          generator=g)
    cache[..., 32 * D:32 * D + 2] = 120
    raw, x = cache[:, heads].cpu().numpy(), src.double().cpu().numpy()
    kept = _kept(slots)
    p8.store(raw, kept, x[:, heads], x[:, [H + h for h in heads]])
    kda.byte_cache_append(src[:, :H], src[:, H:], torch.tensor(slots, device=DEV), cache)
    assert kda.get_device_error() == (5 if kept != slots else 0)
    got = cache[:, heads].cpu().numpy()
    assert np.array_equal(got[..., 32 * D:], raw[..., 32 * D:])
    assert np.array_equal(p8.value(got[..., :32 * D]), p8.value(raw[..., :32 * D]))


@pytest.mark.parametrize("slots", [
    [0, -1, 1], [3, 17, 4], [0, 16, 1, 17, 2, 18], [16, 17, -1, -1, 18, 40],
    list(range(16, 32)) + [5, 0], [5] + list(range(16, 31)) + [6, 7],
    list(range(15)) + [30, 15, 31], [2, 33, 50, 3, 34, 51, 70]])
def test_a_block_met_again(slots):
    _check(slots, 2, 64, torch.bfloat16)


def test_blocks_of_their_own_are_not_reported():
    """The same places of other blocks, none, and a whole block between them."""
    _check([5] + list(range(16, 32)) + [40, 41, -1, 90, 75, 60], 2, 64, torch.bfloat16)


def test_slots_outside_the_cache_are_of_no_block():
    """Not of the block either that their number is in 32 bits of."""
    cache = torch.zeros((1, 1, 1, 32 * 64 + 16), dtype=torch.uint8, device=DEV)
    x = torch.ones((3, 1, 64), device=DEV)
    slots = torch.tensor([(1 << 36) + 2, -5, 3], device=DEV)
    kda.byte_cache_append(x, x, slots, cache)
    assert kda.get_device_error() == 5
    k, v = kda.byte_cache_read(slots[2:], cache, torch.float32)
    assert (k == 1).all() and (v == 1).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,H,T", [(64, 3, 200), (128, 2, 77), (128, 8, 1600), (64, 8, 1600),
                                   (128, 24, 5600), (64, 24, 5600)])
def test_batches_in_any_order(dtype, D, H, T):
    """A few tokens, a warp for each and head; more; as many as make a warp take a window."""
    rng = np.random.RandomState(T + D)
    blocks = T // 2 + 40
    _check(_pieces(rng, T, blocks), H, D, dtype, blocks=blocks, heads=[0, H - 1])
