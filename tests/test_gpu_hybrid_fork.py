"""The hybrid serving example with requests that go on as several and a cache of either form."""
import pytest
import torch

import linear_attention_layer_gb300 as kda
from tests.test_gpu_hybrid_example import _device, _module  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8])
def test_answers_go_on_as_on_a_server_of_their_own(bits):
    """Two prompts, one of them forked into three answers, ends, a compaction in between: each
    row's outputs are those of a server that fed it the same tokens alone.  The calls compute the
    same values in another order of sums: bf16 roundings of layer outputs, 1e-2 each, of a
    residual stream of four layers."""
    ex = _module()
    model = ex.HybridModel(blocks=1)

    def tokens(n):
        return torch.randn((n, 512), device="cuda").to(torch.bfloat16)

    server = ex.Server(model, slots=4, pages=40, page_size=16, max_blocks=8, bits=bits)
    prompts = [tokens(37), tokens(20)]
    fed = [[prompts[0]], [prompts[1]], [], []]
    outs = [None] * 4

    def step(new):
        xs = [tokens(n) if n else None for n in new]
        out = server.step(torch.cat([x for x in xs if x is not None]), new).split(new)
        for b, x in enumerate(xs):
            if x is not None:
                fed[b].append(x)
                outs[b] = out[b]

    server.step(torch.cat(prompts), [37, 20, 0, 0])
    server.fork([0, 0, 0, 1])
    fed = [list(fed[p]) for p in (0, 0, 0, 1)]
    step([1, 1, 1, 1])
    step([1, 0, 5, 1])
    server.compact()
    step([1, 1, 1, 1])
    server.fork([2, -1, 2, 1])
    fed = [list(fed[2]), [], list(fed[2]), list(fed[1])]
    step([1, 0, 1, 1])
    assert kda.get_device_error() == 0
    assert server.held.tolist() == [sum(len(x) for x in f) for f in fed]
    for b in (0, 2, 3):
        alone = ex.Server(model, slots=1, pages=8, page_size=16, max_blocks=8, bits=bits)
        for x in fed[b]:
            want = alone.step(x, [len(x)])
        rel = (outs[b].float() - want.float()).norm() / want.float().norm()
        assert rel <= 4e-2, (b, float(rel))
    server.fork([-1] * 4)
    head, tail = server.free_range.tolist()
    assert tail - head == 40 and server.held.tolist() == [0] * 4
