"""GPU tests of the 8-bit cache's calls and those on shared pages right behind other work: their
kernels may start before what is ahead of them has ended, and have to wait for it.  Nothing here
waits on the host between the calls that are tested; what a call reads is wrong until just before."""
import numpy as np
import pytest
import torch

import linear_attention_layer_gb300 as kda
from tests.test_gpu_cache import DEV, _device, i32  # noqa: F401 (a fixture)
from tests.test_oracle_byte_cache import _random_state

pytestmark = pytest.mark.gpu

GROUP = 32 * 128 + 16


def _randn(g, *shape):
    return torch.randn(shape, device=DEV, generator=g).bfloat16()


class Chain:
    """Append, read, append, attention on a cache of its own, one after the other: a prompt, then
    ``new`` tokens of each request that raise their blocks' exponents."""

    def __init__(self, seed, new):
        g = torch.Generator(device=DEV).manual_seed(seed)
        H, P, B, L, most = 8, 32, 3, 1701, 64
        self.new, blocks = new, -(-(L + most) // P)
        self.cache = torch.empty((B * blocks, H, P // 16, GROUP), dtype=torch.uint8, device=DEV)
        self.table = torch.randperm(B * blocks, device=DEV, generator=g).int().view(B, blocks)

        def slots(lo, hi):
            t = torch.arange(lo, hi, device=DEV)
            return (self.table[:, t // P].long() * P + t % P).flatten()

        self.k, self.v = _randn(g, 2, B * L, H, 128)
        self.k2, self.v2 = 300 * _randn(g, 2, B * new, H, 128)
        self.q = _randn(g, B * new, 16, 128) * 0.01
        self.slots, self.slots2 = slots(0, L), slots(L, L + new)
        self.lens, self.cu = i32([L + new] * B), i32(np.arange(B + 1) * new)
        self.outs = [torch.empty_like(self.k), torch.empty_like(self.v), torch.empty_like(self.q),
                     torch.empty((B * new, 16), device=DEV)]
        self.ws = torch.empty(kda.byte_cache_attention_workspace_size(
            self.cache, B, B * new, 16, new, blocks, torch.bfloat16), dtype=torch.uint8, device=DEV)

    def poison(self):
        self.cache.fill_(120)
        for x in self.outs:
            x.fill_(-7)

    def run(self, between=lambda: None, **kw):
        kda.byte_cache_append(self.k, self.v, self.slots, self.cache, **kw)
        between()
        kda.byte_cache_read(self.slots, self.cache, k=self.outs[0], v=self.outs[1], **kw)
        between()
        kda.byte_cache_append(self.k2, self.v2, self.slots2, self.cache, **kw)
        between()
        kda.byte_cache_attention(self.q, self.cache, self.table, self.lens, self.cu,
                                 max_new=self.new, out=self.outs[2], lse=self.outs[3],
                                 workspace=self.ws, **kw)

    def result(self):
        torch.cuda.synchronize()
        return [x.clone() for x in (*self.outs, self.cache)]

    def one_by_one(self):
        self.poison()
        self.run(torch.cuda.synchronize)
        return self.result()


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("new", [1, 3, 60])
def test_calls_behind_one_another(new):
    """On the current stream, on one passed in, and captured."""
    c = Chain(new, new)
    want = c.one_by_one()
    assert (want[2].float().abs() > 0).all() and kda.get_device_error() == 0
    for _ in range(3):
        c.poison()
        c.run()
        assert _same(c.result(), want)
    side = torch.cuda.Stream()
    c.poison()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    assert _same(c.result(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for _ in range(3):
        c.poison()
        torch.cuda.synchronize()
        g.replay()
        assert _same(c.result(), want)


def test_chains_on_two_streams_at_once():
    chains = [Chain(1, 1), Chain(2, 60)]
    want = [c.one_by_one() for c in chains]
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(5):
        for c in chains:
            c.poison()
        torch.cuda.synchronize()
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                c.run()
        for c, w in zip(chains, want):
            assert _same(c.result(), w)


def test_graphs_of_chains_that_share_a_workspace():
    chains = [Chain(3, 1), Chain(4, 60)]
    want = [c.one_by_one() for c in chains]
    ws = max((c.ws for c in chains), key=lambda w: w.numel())
    graphs = []
    for c in chains:
        c.ws = ws
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 1)):
        for c in chains:
            c.poison()
        ws.fill_(0xff)
        torch.cuda.synchronize()
        for i in order:
            graphs[i].replay()
        for c, w in zip(chains, want):
            assert _same(c.result(), w)


# ------------------------------------ an input written by the node right ahead ---

def _copy():
    g = torch.Generator(device=DEV).manual_seed(0)
    caches = [torch.randint(0, 256, (8, 2, 2, GROUP), dtype=torch.uint8, device=DEV, generator=g)
              for _ in range(2)]
    start = [c.clone() for c in caches]

    def reset():
        for c, s in zip(caches, start):
            c.copy_(s)
    copies = i32([[0, 5, 32], [1, 6, 17]])
    return copies, i32([[0, 7, 32], [2, 4, 32]]), lambda: kda.cache_copy(caches, copies), caches, reset


def _copied_pages():
    """The pages copied from are what the node ahead writes."""
    pages = torch.zeros((4, 2, 2, GROUP), dtype=torch.uint8, device=DEV)
    cache = torch.zeros_like(pages)  # the first half of it is written
    copies = i32([[0, 2, 32], [1, 3, 17]])
    half, wrong = cache[:2], pages[:2].clone()
    half.random_(0, 255, generator=torch.Generator(device=DEV).manual_seed(1))
    wrong.fill_(77)
    return half, wrong, lambda: kda.cache_copy([cache], copies), [cache], lambda: cache[2:].fill_(9)


def _fork():
    rng = np.random.RandomState(5)
    held, table, ring, span = _random_state(rng, 6, 16, 4, 40)
    parents, keep = i32([0, 0, 1, 3, 3, 5, -1]), i32([min(held)] * 7)
    args = [i32(held), i32(table), parents, keep]
    free, span = i32(ring), torch.tensor(span, device=DEV)
    kept, outs = free.clone(), [torch.empty(n, dtype=t, device=DEV) for n, t in (
        ((7,), torch.int32), ((7, 4), torch.int32), ((7, 3), torch.int32), ((2,), torch.int64))]

    def run():
        kda.cache_fork(*args, free, span, page_size=16, num_pages=40, kv_lens=outs[0],
                       block_table_out=outs[1], copies=outs[2], free_range_out=outs[3])

    def reset():
        free.copy_(kept)
    return parents, i32([2, 4, -1, -1, 0, 1, 5]), run, [*outs, free], reset


def _compact():
    held, table, ring, _ = _random_state(np.random.RandomState(5), 9, 16, 5, 60)
    lens, table, free = i32(held), i32(table), i32(ring)
    kept = free.clone()  # (entries past the free pages stay as they are)
    outs = [torch.empty(n, dtype=t, device=DEV) for n, t in (
        ((9, 5), torch.int32), ((30, 3), torch.int32), ((2,), torch.int64))]

    def run():
        kda.cache_compact(lens, table, free, page_size=16, num_pages=60, block_table_out=outs[0],
                          copies=outs[1], free_range_out=outs[2])
    return lens, (lens // 2).int(), run, [*outs, free], lambda: free.copy_(kept)


def _append():
    c = Chain(7, 1)
    return (c.k, c.k.flip(0).contiguous(),
            lambda: kda.byte_cache_append(c.k, c.v, c.slots, c.cache), [c.cache], c.poison)


def _read():
    c = Chain(8, 1)
    c.one_by_one()
    return (c.slots, c.slots.flip(0).contiguous(),
            lambda: kda.byte_cache_read(c.slots, c.cache, k=c.outs[0], v=c.outs[1]), c.outs[:2],
            lambda: [x.fill_(-7) for x in c.outs[:2]])


def _attention(new):
    c = Chain(9, new)
    c.one_by_one()
    return (c.lens, c.lens - 1000, lambda: kda.byte_cache_attention(
        c.q, c.cache, c.table, c.lens, c.cu, max_new=new, out=c.outs[2], lse=c.outs[3],
        workspace=c.ws), c.outs[2:], lambda: [x.fill_(-7) for x in c.outs[2:]])


CALLS = dict(copy=_copy, copied_pages=_copied_pages, fork=_fork, compact=_compact, append=_append,
             read=_read, attention=lambda: _attention(1), chunk=lambda: _attention(60))


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("ahead", ["a kernel", "a copy", "a kernel of another stream"])
def test_a_call_waits_for_the_node_ahead(call, ahead):
    """Captured right behind long work and the node that writes one of its inputs, which holds
    other, valid values when a replay begins."""
    given, other, run, outs, reset = CALLS[call]()
    right, room = given.clone(), torch.zeros(1 << 26, device=DEV)
    reset()
    run()
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    side = torch.cuda.Stream()

    def write():
        for _ in range(4):
            room.add_(1)
        if ahead == "a copy":
            given.copy_(right)
        else:
            torch.maximum(right, right, out=given)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cur = torch.cuda.current_stream()
        if ahead == "a kernel of another stream":
            side.wait_stream(cur)
            with torch.cuda.stream(side):
                write()
            cur.wait_stream(side)
        else:
            write()
        run()
    reset()
    given.copy_(other)
    run()
    torch.cuda.synchronize()
    assert not _same(outs, want)  # the other values would show
    for _ in range(3):
        reset()
        given.copy_(other)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert _same(outs, want)
    reset()
    given.copy_(other)
    torch.cuda.synchronize()
    write()
    run()
    torch.cuda.synchronize()
    assert _same(outs, want)


def test_a_copy_behind_a_memset():
    """The pages copied from are what a memset leaves."""
    cache = torch.empty((4, 2, 2, GROUP), dtype=torch.uint8, device=DEV)
    copies, room = i32([[0, 2, 32], [1, 3, 17]]), torch.zeros(1 << 26, device=DEV)
    kda.cache_copy(cache.zero_(), i32([[-1, -1, 0]]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(4):
            room.add_(1)
        cache[:2].zero_()
        kda.cache_copy(cache, copies)
    for _ in range(3):
        cache.fill_(99)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert not cache[:3].any() and not cache[3, :, :2].any()


# ------------------------------------------------ results that repeat themselves ---

@pytest.mark.parametrize("kv,new,heads", [([2048], [1], 32), ([300, 8000, 4001] * 20, [1] * 60, 32),
                                          ([60001], [1], 32), ([5000], [700], 32),
                                          ([900, 70, 33], [60, 1, 3], 8)])
def test_attention_repeats_itself(kv, new, heads):
    """Bit for bit, whatever the workspace and the outputs held before."""
    g = torch.Generator(device=DEV).manual_seed(sum(kv))
    H, P = 8, 64
    need = [-(-n // P) for n in kv]
    pages = sum(need)
    cache = torch.empty((pages, H, P // 16, GROUP), dtype=torch.uint8, device=DEV)
    kv_all = _randn(g, 2, pages * P, H, 128)
    kda.byte_cache_append(kv_all[0], kv_all[1], torch.arange(pages * P, device=DEV), cache)
    ids, table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)), []
    for n in need:
        table.append(ids[:n].tolist() + [-1] * (max(need) - n))
        ids = ids[n:]
    args = i32(table), i32(kv), i32(np.concatenate([[0], np.cumsum(new)]))
    q = _randn(g, sum(new), heads, 128)
    ws = torch.empty(kda.byte_cache_attention_workspace_size(
        cache, len(kv), sum(new), heads, max(new), max(need), torch.bfloat16), dtype=torch.uint8,
        device=DEV)
    first = None
    for fill in (0, 0xff, 0x7f, 1, 0x80):
        ws.fill_(fill)
        out = torch.full_like(q, float(fill))
        o, lse = kda.byte_cache_attention(q, cache, *args, max_new=max(new), out=out,
                                          return_lse=True, workspace=ws)
        first = first or (o.clone(), lse.clone())
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    assert first[0].isfinite().all() and kda.get_device_error() == 0
