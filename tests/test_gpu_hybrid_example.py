"""The hybrid serving example: the cache calls and the KDA calls in one model's steps."""
import pytest
import torch

import linear_attention_layer_gb300 as kda

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def _module():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "hybrid_serving.py")
    spec = importlib.util.spec_from_file_location("hybrid_serving", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs():
    assert _module().main() == 0


def test_chunks_and_single_tokens_give_what_whole_prompts_give():
    """The same tokens in one step, in chunks and one at a time.  The cache quantises each
    token alike, so the runs differ by the bf16 rounding of layer outputs and by how the KDA
    kernels order their sums: 1e-2 each, of a residual stream of four layers."""
    ex = _module()
    model = ex.HybridModel(blocks=1)
    lens = [70, 33]
    x = [torch.randn((n, 512), device="cuda").to(torch.bfloat16) for n in lens]
    whole = ex.Server(model, slots=2, pages=8, page_size=16, max_blocks=8)
    want = whole.step(torch.cat(x), lens).float().split(lens)
    parts = ex.Server(model, slots=2, pages=8, page_size=16, max_blocks=8)
    got = [[], []]
    at = [0, 0]
    for new in ([40, 20], [29, 5], [0, 7], [1, 1]):
        step = torch.cat([x[b][at[b]:at[b] + new[b]] for b in range(2)])
        out = parts.step(step, new).float().split(new)
        for b in range(2):
            got[b].append(out[b])
            at[b] += new[b]
    assert kda.get_device_error() == 0
    assert parts.held.tolist() == lens == whole.held.tolist()
    for b in range(2):
        y = torch.cat(got[b])
        rel = (y - want[b]).norm() / want[b].norm()
        assert rel <= 4e-2, (b, float(rel))


def test_a_slot_is_clean_for_its_next_request():
    """A request ends and another starts in its slot: its outputs are those of a server on which
    the slot was never used, bit for bit: the same calls on the same values, in other pages."""
    ex = _module()
    model = ex.HybridModel(blocks=1)

    def tokens(n):
        return torch.randn((n, 512), device="cuda").to(torch.bfloat16)

    first, other, second = tokens(50), [tokens(n) for n in (20, 1, 1, 1)], [tokens(33), tokens(1)]
    used, fresh = (ex.Server(model, slots=2, pages=12, page_size=16, max_blocks=8)
                   for _ in range(2))
    used.step(torch.cat([first, other[0]]), [50, 20])
    used.step(other[1], [-1, 1])
    fresh.step(other[0], [0, 20])
    fresh.step(other[1], [0, 1])
    for i, n in enumerate((33, 1)):
        a, b = (s.step(torch.cat([second[i], other[2 + i]]), [n, 1])[:n] for s in (used, fresh))
        assert torch.equal(a, b), i
    assert used.held.tolist() == fresh.held.tolist() == [34, 23]
    assert kda.get_device_error() == 0
