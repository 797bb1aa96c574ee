"""GPU tests of pages that several rows hold (fork, compact, copy) against the oracle's loops:
everything is whole numbers and bytes, compared exactly."""
import numpy as np
import pytest
import torch

import linear_attention_layer_gb300 as kda
from oracle import byte_cache as p8
from tests.test_gpu_cache import DEV, _device, i32  # noqa: F401 (a fixture)
from tests.test_oracle_byte_cache import _random_state

pytestmark = pytest.mark.gpu


def _i64(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def _fork(held, table, parents, keep, ring, span, P, N, **kw):
    r = i32(ring)
    kv, out, copies, sp = kda.cache_fork(i32(held), i32(table), i32(parents), i32(keep), r,
                                         _i64(span), page_size=P, num_pages=N, **kw)
    return [x.cpu().numpy() for x in (kv, out, copies, sp, r)]


def _check_fork(held, table, parents, keep, ring, span, P, N, **kw):
    got = _fork(held, table, parents, keep, ring, span, P, N, **kw)
    *want, err = p8.fork(held, np.asarray(table), parents, keep, ring, span, P, N)
    want[2] = np.array(want[2]).reshape(-1, 3)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert kda.get_device_error() == (5 if err else 0)
    return got


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("B,R,N", [(1, 8, 20), (7, 11, 60), (40, 0, 200), (0, 3, 5), (60, 300, 700)])
def test_fork(seed, B, R, N):
    rng = np.random.RandomState(seed)
    held, table, ring, span = _random_state(rng, B, 16, 5, N)
    parents = rng.randint(-1, B, R) if B else np.full(R, -1)
    keep = [int(rng.choice([held[p], rng.randint(0, held[p] + 1)])) if p >= 0 else 0
            for p in parents]
    _check_fork(held, table, parents, keep, ring, span, 16, N)


@pytest.mark.parametrize("B,R,blocks,N", [(60, 300, 30, 700), (9, 1024, 5, 900), (9, 1025, 5, 900),
                                          (40, 40, 100, 65536), (40, 40, 100, 65537),
                                          (300, 400, 374, 1300), (300, 400, 376, 1300)])
def test_fork_at_the_borders_of_its_forms(B, R, blocks, N):
    """One CTA, one cluster and a kernel a step: by entries of the tables, rows and pages."""
    for seed in range(3):
        rng = np.random.RandomState(seed)
        held, table, ring, span = _random_state(rng, B, 16, blocks, N)
        parents = rng.randint(-1, B, R)
        keep = [int(rng.choice([held[p], rng.randint(0, held[p] + 1)])) if p >= 0 else 0
                for p in parents]
        need = sum(1 for k in keep if k % 16)
        if need > span[1] - span[0]:
            keep = [k // 16 * 16 if i % 4 else k for i, k in enumerate(keep)]
        _check_fork(held, table, parents, keep, ring, span, 16, N)


@pytest.mark.parametrize("R,rows", [(2500, 3), (3, 2500)])
def test_fork_of_many_rows_and_long_ones(R, rows):
    """More rows than a pass of the CTA that settles them, rows of more columns than a CTA takes,
    more pages than its threads have words at once."""
    rng = np.random.RandomState(R)
    P, blocks, N = 16, 2100, 70000
    ids = list(rng.permutation(N))
    table, held = np.full((rows, blocks), -1), []
    for b in range(rows):
        n = 2090 - b % 7 if rows == 3 else rng.randint(0, 20)
        for c in range(n):
            table[b, c] = table[0, c] if b and c < n // 2 and c < -(-held[0] // P) - 1 else ids.pop()
        held.append(max(0, n * P - rng.randint(0, P)))
    ring = np.full(N, -1)
    ring[:len(ids)] = ids
    parents = rng.randint(0, rows, R)
    keep = [int(rng.choice([held[p], rng.randint(0, held[p] + 1)])) for p in parents]
    _check_fork(held, table, parents, keep, ring, (0, len(ids)), P, N)


def test_fork_refusals():
    P, N = 16, 8
    table, held, ring = np.array([[3, 1, -1], [5, -1, -1]]), [20, 9], np.array([0, 2, 4, 6, 7, 0, 0, 0])

    def go(parents, keep, held=held, table=table, span=(0, 5)):
        return _check_fork(held, table, parents, keep, ring, span, P, N)
    go([2, -2, 0, 1 << 30], [1, 1, 20, 0])             # parents out of range
    go([0, 0, 1, 1], [21, -1, 9, 10])                  # lengths out of range
    go([0, 0, 0, 0, 1], [20, 20, 20, 16, 9], span=(0, 2))  # two pages for three copies... enough
    go([0, 0, 0, 0, 1, 1], [20, 20, 20, 20, 9, 9], span=(3, 5))  # too few pages
    for span in ((-1, 2), (3, 2), (0, 9)):             # a malformed ring is an empty one
        go([0, 0], [20, 20], span=span)
    for bad in ([-1, 9], [49, 9]):                     # rows that make no sense keep their pages
        go([0, 1, 1], [3, 9, 9], held=bad)
    bad = table.copy()
    bad[0, 0], bad[1, 0] = 8, -5                       # page indexes outside the cache
    go([0, 0, 1], [20, 20, 9], table=bad)
    go([0, 0], [20, 7], table=bad)


def test_fork_in_place_and_callers_workspace():
    rng = np.random.RandomState(2)
    held, table, ring, span = _random_state(rng, 6, 16, 5, 60)
    parents = rng.randint(0, 6, 9)
    keep = [held[p] for p in parents]
    base = _fork(held, table, parents, keep, ring, span, 16, 60)
    size = kda.cache_fork_workspace_size(60, 9)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
    k, r, sp = i32(keep), i32(ring), _i64(span)
    out = torch.full((9, 5), 77, dtype=torch.int32, device=DEV)
    cp = torch.full((9, 3), 77, dtype=torch.int32, device=DEV)
    kv, o, c, s = kda.cache_fork(i32(held), i32(table), i32(parents), k, r, sp, page_size=16,
                                 num_pages=60, kv_lens=k, block_table_out=out, copies=cp,
                                 free_range_out=sp, workspace=ws)
    assert kv is not None and o.data_ptr() == out.data_ptr() and s.data_ptr() == sp.data_ptr()
    for a, b in zip(base, (kv, o, c, s, r)):
        assert np.array_equal(a, b.cpu().numpy())
    for bad in (dict(workspace=ws[:-256]), dict(block_table_out=i32(table)[:0])):
        with pytest.raises((kda.KDAError, ValueError)):
            kda.cache_fork(i32(held), i32(table), i32(parents), i32(keep), i32(ring), _i64(span),
                           page_size=16, num_pages=60, **bad)


def _check_compact(held, table, ring, P, N, **kw):
    r = i32(ring)
    out, copies, span = kda.cache_compact(i32(held), i32(table), r, page_size=P, num_pages=N, **kw)
    *want, err = p8.compact(held, np.asarray(table), ring, P, N)
    want[1] = np.array(want[1]).reshape(-1, 3)
    for g, w in zip((out, copies, span, r), want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert kda.get_device_error() == (5 if err else 0)


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("B,N", [(1, 4), (9, 60), (0, 7), (64, 256), (200, 1024)])
def test_compact(seed, B, N):
    rng = np.random.RandomState(seed)
    held, table, ring, _ = _random_state(rng, B, 16, 5, N)
    _check_compact(held, table, ring, 16, N)


@pytest.mark.parametrize("B,blocks,N", [(64, 30, 256), (64, 34, 256), (200, 50, 1024),
                                        (40, 100, 65536), (40, 100, 65537), (300, 873, 1300),
                                        (300, 875, 1300)])
def test_compact_at_the_borders_of_its_forms(B, blocks, N):
    for seed in range(3):
        rng = np.random.RandomState(seed)
        held, table, ring, _ = _random_state(rng, B, 16, blocks, N)
        _check_compact(held, table, ring, 16, N)


@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 64])
def test_compact_of_full_and_nearly_full_caches(N):
    rng = np.random.RandomState(N)
    for live in {0, 1, N // 2, N - 1, N}:
        table = np.full((1, N + 1), -1)
        table[0, :live] = rng.permutation(N)[:live]
        _check_compact([live * 16], table, np.full(N, -3), 16, N)


def test_compact_of_many_pages():
    rng = np.random.RandomState(1)
    N, B, blocks = 200003, 50, 3000
    ids = rng.permutation(N)
    table = ids[:B * blocks].reshape(B, blocks)
    held = [int(x) for x in rng.randint(0, blocks * 16 + 1, B)]
    _check_compact(held, table, np.zeros(N, int), 16, N)


def test_compact_refusals_and_in_place():
    ring = np.zeros(8, int)
    table = np.array([[3, 7, -1], [5, -1, -1]])
    _check_compact([-1, 9], table, ring, 16, 8)
    _check_compact([49, 9], table, ring, 16, 8)
    bad = table.copy()
    bad[0, 0] = 8
    _check_compact([20, 9], bad, ring, 16, 8)
    t = i32(table)
    out, _, _ = kda.cache_compact(i32([20, 9]), t, i32(ring), page_size=16, num_pages=8,
                                  block_table_out=t)
    assert out.data_ptr() == t.data_ptr()
    assert t.tolist() == p8.compact([20, 9], table, ring, 16, 8)[0].tolist()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D,H,P,layers", [(128, 8, 64, 1), (64, 1, 16, 3), (128, 3, 48, 70),
                                          (64, 2, 256, 2), (128, 5, 4096, 1)])
def test_copy(bits, D, H, P, layers):
    rng = np.random.RandomState(D + H)
    N = 9 if P < 4096 else 4
    size = 18 * D if bits == 4 else 32 * D + 16
    caches = [torch.randint(0, 256, (N, H, P // 16, size), dtype=torch.uint8, device=DEV)
              for _ in range(layers)]
    ids = rng.permutation(N)
    copies = [[int(ids[0]), int(ids[1]), P], [-1, -1, 0], [int(ids[2]), int(ids[3]), 1]]
    if N > 4:
        copies += [[int(ids[0]), int(ids[4]), P - 15], [int(ids[2]), int(ids[5]), 16],
                   [int(ids[0]), int(ids[6]), min(P, 17)], [int(ids[7]), int(ids[7]), P],
                   [int(ids[7]), int(ids[8]), 0]]
    want = [c.cpu().numpy() for c in caches]
    for w in want:
        p8.copy(w, copies)
    kda.cache_copy(caches, i32(copies))
    for c, w in zip(caches, want):
        assert np.array_equal(c.cpu().numpy(), w)


def test_copies_out_of_range_are_skipped():
    cache = torch.randint(0, 256, (4, 2, 2, 2064), dtype=torch.uint8, device=DEV)
    before = cache.clone()
    for bad in ([4, 0, 16], [0, 4, 16], [-2, 0, 16], [0, -1, 16], [0, 1, 33], [0, 1, -1]):
        kda.cache_copy(cache, i32([bad]))
        assert kda.get_device_error() == 5 and torch.equal(cache, before)
    kda.cache_copy([], i32([[0, 1, 16]]))
    kda.cache_copy(cache, i32(np.zeros((0, 3))))
    assert torch.equal(cache, before)


def test_graph_and_side_stream():
    """Captured with its copies and replayed on other lengths, and on another stream."""
    P, N = 16, 40
    rng = np.random.RandomState(4)
    held, table, ring, span = _random_state(rng, 6, P, 4, N)
    parents = [0, 0, 1, 3, 3, 5, -1]
    args = [i32(held), i32(table), i32(parents), i32([0] * 7), i32(ring), _i64(span)]
    cache = torch.randint(0, 256, (N, 2, 1, 2064), dtype=torch.uint8, device=DEV)

    def go():
        res = kda.cache_fork(*args, page_size=P, num_pages=N)
        kda.cache_copy(cache, res[2])
        return res
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = go()
    for keep in ([held[p] if p >= 0 else 0 for p in parents],
                 [max(0, held[p] - 5) if p >= 0 else 0 for p in parents]):
        args[3].copy_(i32(keep))
        args[4].copy_(i32(ring))
        before = cache.cpu().numpy()
        g.replay()
        torch.cuda.synchronize()
        kv, out, copies, sp, rg, _ = p8.fork(held, table, parents, keep, ring, span, P, N)
        for a, b in zip(res, (kv, out, copies, sp)):
            assert np.array_equal(a.cpu().numpy(), np.array(b))
        assert np.array_equal(args[4].cpu().numpy(), rg)
        p8.copy(before, copies)
        assert np.array_equal(cache.cpu().numpy(), before)


@pytest.mark.parametrize("where", ["first", "after a memset", "after another stream",
                                   "on another stream"])
def test_copy_captured_behind_anything(where):
    """The copies' kernel may start before what is ahead of it has ended: as a graph's first node,
    behind a memset or kernels of its own stream and of another one it still waits for them."""
    caches = [torch.randint(0, 256, (8, 2, 2, 2064), dtype=torch.uint8, device=DEV)
              for _ in range(2)]
    copies, room = i32([[0, 5, 32], [1, 6, 17]]), torch.zeros(1 << 22, device=DEV)
    given = copies.clone()
    side = torch.cuda.Stream()
    kda.cache_copy(caches, copies)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cur = torch.cuda.current_stream()
        if where == "after a memset":
            copies.zero_()
            copies.copy_(given)
            room.zero_()
        elif where == "after another stream":
            side.wait_stream(cur)
            with torch.cuda.stream(side):
                copies.zero_()
                for _ in range(20):
                    room.add_(1)
                copies.copy_(given)
            cur.wait_stream(side)
        if where == "on another stream":
            side.wait_stream(cur)
            kda.cache_copy(caches, copies, stream=side)
            cur.wait_stream(side)
        else:
            kda.cache_copy(caches, copies)
    for _ in range(3):
        for c in caches:
            c[5:].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for c in caches:
            assert torch.equal(c[5], c[0]) and torch.equal(c[6], c[1]) and not c[7].any()


def test_graphs_that_share_a_workspace():
    """A fork and a compaction captured with one workspace and replayed in turn, on a side stream."""
    P, N = 16, 60
    rng = np.random.RandomState(5)
    held, table, ring, span = _random_state(rng, 7, P, 5, N)
    parents = [0, 0, 1, 3, 3, 5, -1, 6]
    keep = [held[p] if p >= 0 else 0 for p in parents]
    ws = torch.full((max(kda.cache_fork_workspace_size(N, 8), kda.cache_compact_workspace_size(N)),),
                    0xff, dtype=torch.uint8, device=DEV)
    h, t, p, k, sp = i32(held), i32(table), i32(parents), i32(keep), _i64(span)
    r1, r2 = i32(ring), i32(ring)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g1, stream=s):
            a = kda.cache_fork(h, t, p, k, r1, sp, page_size=P, num_pages=N, workspace=ws)
        with torch.cuda.graph(g2, stream=s):
            b = kda.cache_compact(h, t, r2, page_size=P, num_pages=N, workspace=ws)
    want_a = p8.fork(held, table, parents, keep, ring, span, P, N)
    want_b = p8.compact(held, table, ring, P, N)
    for _ in range(3):
        for x in (*a, *b):
            x.fill_(-7)
        r1.copy_(i32(ring)), r2.copy_(i32(ring))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g1.replay()
            g2.replay()
        torch.cuda.synchronize()
        for x, w in zip((*a, r1), want_a):
            assert np.array_equal(x.cpu().numpy(), np.array(w))
        for x, w in zip((*b, r2), want_b):
            assert np.array_equal(x.cpu().numpy(), np.array(w))


@pytest.mark.parametrize("bits", [4, 8])
def test_a_server_forks_and_compacts(bits):
    """Prompts, several answers each, beams, ends and a compaction into fewer pages: after every
    step each row's attention is what it is over a cache of its own, bit for bit."""
    P, Hk, Hq, D, pages = 16, 2, 4, 64, 80
    rng = np.random.RandomState(bits)
    empty, append, attention, read = (
        (kda.cache_empty, kda.cache_append, kda.cache_attention, kda.cache_read) if bits == 4 else
        (kda.byte_cache_empty, kda.byte_cache_append, kda.byte_cache_attention, kda.byte_cache_read))
    caches = [empty(pages, P, Hk, D, DEV) for _ in range(2)]
    table = torch.full((3, 8), -1, dtype=torch.int32, device=DEV)
    ring = torch.arange(pages, dtype=torch.int32, device=DEV)
    span = _i64([0, pages])
    lens = i32([0, 0, 0])
    history = [[], [], []]  # tokens of each row, by seed

    def token(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        return torch.randn((3, 1, Hk, D), device=DEV, generator=g).bfloat16()

    def check():
        B = len(history)
        q = torch.randn((B, Hq, D), device=DEV).bfloat16()
        cu = i32(np.arange(B + 1))
        used = [h for h in history]
        for layer, cache in enumerate(caches):
            got = attention(q, cache, table, lens, cu, max_new=1)
            for b, h in enumerate(used):
                if not h:
                    assert not got[b].any()
                    continue
                own = empty(-(-len(h) // P), P, Hk, D, DEV)
                for t, seed in enumerate(h):  # in the order of the steps: exponents rise alike
                    x = token(seed)[layer:layer + 2]
                    append(x[0], x[1], _i64([t]), own)
                row = torch.arange(own.shape[0], dtype=torch.int32, device=DEV)[None]
                want = attention(q[b:b + 1], own, row, i32([len(h)]), i32([0, 1]), max_new=1)
                assert torch.equal(got[b], want[0]), (b, layer)

    def feed(new):
        nonlocal lens, span
        seeds = [[int(rng.randint(1 << 30)) for _ in range(max(n, 0))] for n in new]
        steps = max([len(s) for s in seeds])
        for i in range(steps):  # one token at a time
            now = [1 if i < len(s) else 0 for s in seeds]
            lens, cu, slots, span = kda.cache_tables(lens, lens, i32(now), table, ring, span,
                                                     page_size=P, max_tokens=sum(now))
            xs = [token(s[i]) for s in seeds if i < len(s)]
            for layer, cache in enumerate(caches):
                append(torch.cat([x[layer] for x in xs]), torch.cat([x[layer + 1] for x in xs]),
                       slots, cache)
        for h, s in zip(history, seeds):
            h += s

    def fork(parents, keep):
        nonlocal lens, span, table, history
        lens, table, copies, span = kda.cache_fork(lens, table, i32(parents), i32(keep), ring, span,
                                                   page_size=P, num_pages=pages)
        kda.cache_copy(caches, copies)
        history = [history[p][:n] if p >= 0 else [] for p, n in zip(parents, keep)]

    def free():
        head, tail = span.tolist()
        return tail - head

    feed([37, 5, 32])
    check()
    fork([0, 0, 0, 1, 2, 2], [37, 37, 37, 5, 32, 32])
    check()
    feed([1, 2, 3, 20, 1, 1])
    check()
    fork([2, 2, 0, 1, -1, 5, 3, 3], [40, 40, 38, 39, 0, 33, 25, 25])
    feed([1, 1, 1, 1, 1, 1, 1, 1])
    check()
    fork([0, 1, 7, 6], [41, 37, 20, 26])  # ends, and some cut back
    feed([2, 1, 1, 0])
    check()
    table, copies, span = kda.cache_compact(lens, table, ring, page_size=P, num_pages=pages)
    kda.cache_copy(caches, copies)
    check()
    live = pages - free()
    assert int(table.max()) == live - 1
    smaller = live + 6  # the cache goes on in fewer pages
    caches = [c[:smaller].clone() for c in caches]
    ring, span = ring[:smaller].contiguous(), _i64([0, smaller - live])
    pages = smaller
    feed([3, 3, 3, 9])
    check()
    fork([-1, -1], [0, 0])
    assert free() == smaller
