"""GPU test of requests that share pages and are cut: drafts behind what is shared by cache_tables,
anything below by cache_fork."""
import numpy as np
import pytest
import torch

import linear_attention_layer_gb300 as kda
from tests.test_gpu_cache import DEV, _device, i32  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

P, H, D, PAGES, BLOCKS = 16, 2, 64, 24, 6


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("prompt", [32, 37])
def test_drafts_behind_shared_pages_and_cuts_into_them(bits, prompt):
    empty, append, read = (
        (kda.cache_empty, kda.cache_append, kda.cache_read) if bits == 4 else
        (kda.byte_cache_empty, kda.byte_cache_append, kda.byte_cache_read))
    cache = empty(PAGES, P, H, D, DEV)
    table = torch.full((1, BLOCKS), -1, dtype=torch.int32, device=DEV)
    ring, span = torch.arange(PAGES, dtype=torch.int32, device=DEV), torch.tensor([0, PAGES], device=DEV)
    lens = i32([0])
    g = torch.Generator(device=DEV).manual_seed(prompt)
    codes = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 4.0], device=DEV)  # both forms hold them exactly
    tokens = []  # of each row

    def step(new, back=0):
        nonlocal lens, span
        lens, cu, slots, span = kda.cache_tables(lens, lens - back, i32(new), table, ring, span,
                                                 page_size=P, max_tokens=sum(new))
        x = codes[torch.randint(0, 6, (sum(new), H, D), device=DEV, generator=g)]
        x[..., ::16] = 6.0  # each block's largest
        append(x, x, slots, cache)
        at = 0
        for b, n in enumerate(new):
            tokens[b] = torch.cat([tokens[b][:len(tokens[b]) - back], x[at:at + n]])
            at += n
        check()

    def fork(parents, keep):
        nonlocal lens, span, table, tokens
        lens, table, copies, span = kda.cache_fork(lens, table, i32(parents), i32(keep), ring, span,
                                                   page_size=P, num_pages=PAGES)
        kda.cache_copy(cache, copies)
        tokens = [tokens[p][:n] for p, n in zip(parents, keep)]
        check()

    def check():
        assert lens.tolist() == [len(t) for t in tokens]
        rows = table.tolist()
        held = {p for r, n in zip(rows, lens.tolist()) for p in r[:-(-n // P)]}
        free = [int(ring[i % PAGES]) for i in range(*span.tolist())]
        assert sorted([*held, *free]) == list(range(PAGES))  # none twice
        for r, t in zip(rows, tokens):
            pos = np.arange(len(t))
            slots = torch.tensor(np.array(r)[pos // P] * P + pos % P, device=DEV)
            for y in read(slots, cache, torch.float32):
                assert torch.equal(y, t)

    tokens.append(torch.zeros((0, H, D), device=DEV))
    step([prompt])
    fork([0, 0, 0], [prompt] * 3)
    step([3, 3, 3])
    step([1, 0, 2], back=3)  # all drafts rejected: back to what is shared
    step([20, 1, 1])
    fork([0, 1, 2], [20, 32, 9])  # cuts into shared pages
    step([5, 1, 8])
    fork([1], [33])
    step([2], back=1)
    assert kda.get_device_error() == 0
