"""GPU tests of the 4-bit paged cache where a call is easily answered wrongly: unusual strides,
long fp32 rows, weights far below the largest, hidden pages, waits that run out."""
import pytest
import torch

import linear_attention_layer_gb300 as kda
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
