"""The 8-bit paged cache of the full-attention layers and the pages that requests share, as
work to be timed.

A server's attention layers keep keys and values in pages.  The operators here hold them in
8 bits, attend over them, and let several requests hold the same pages:

    append8     new k, v into the pages, a scale for each block of 16 tokens and head, and
                the values of the blocks read back
    attend8     queries over the paged cache (one token, windows, chunks)
    fork        new requests from the pages of old ones (beams, several answers to a prompt),
                pages that nobody holds any more given back, unfinished last pages copied
    compact     the pages in use moved to the lowest numbers

Cache format (E4M3 codes, a power of two for K and for V of each block of 16 tokens and head), a
uint8 tensor [num_pages, kv heads, page_size / 16, 32 D + 16].  The bytes of 16 tokens:
    K codes    16 D bytes  [D / 64][16 tokens][4][16]: channel c at [c % (D/4) / 16][i][c / (D/4)][c % 16]
    V codes    16 D bytes  [2][2][8][4][D / 8]: token 8 a + 2 t + b, channel g D/8 + r at [a][b][g][t][r]
    2 bytes    exponents of K and V plus 127, then 14 unused
"""
import math
import zlib

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LEAST = -100  # exponent of a block of zeros


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # The new tokens of a decode step of 256 requests, into blocks begun earlier.
        dict(name="append8_decode_256", op="append8", tokens=256, kv_heads=8, dim=128, page=64,
             dtype="bf16", order="scattered"),
        # An fp32 model's ragged chunk, small heads.
        dict(name="append8_fp32_1237", op="append8", tokens=1237, kv_heads=3, dim=64, page=16,
             dtype="fp32", order="runs"),
        # A packed prefill: 64 sequences of 4224 tokens on average.
        dict(name="append8_prefill_270336", op="append8", tokens=270336, kv_heads=8, dim=128,
             page=64, dtype="bf16", order="runs"),
        # One user, one token, a short conversation: latency.
        dict(name="attend8_1x2048", op="attend8", seqs=1, lo=2048, hi=2048, new_lo=1, new_hi=1,
             heads=32, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # The decode step of the 256-request server.
        dict(name="attend8_decode_256", op="attend8", seqs=256, lo=256, hi=8192, new_lo=1,
             new_hi=1, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # fp32, drafted windows over ragged contexts, some of them empty.
        dict(name="attend8_fp32_67", op="attend8", seqs=67, lo=0, hi=4001, new_lo=1, new_hi=5,
             heads=12, kv_heads=4, dim=64, page=32, dtype="fp32"),
        # One long document, one token.
        dict(name="attend8_long_1x262144", op="attend8", seqs=1, lo=262144, hi=262144, new_lo=1,
             new_hi=1, heads=32, kv_heads=8, dim=128, page=256, dtype="bf16"),
        # A prefill chunk of a long prompt: 2048 new tokens on 30720 cached ones.
        dict(name="attend8_chunk_2048", op="attend8", seqs=1, lo=32768, hi=32768, new_lo=2048,
             new_hi=2048, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # Eight answers to one prompt: latency.
        dict(name="fork_answers_8", op="fork", groups=1, old=1, rows=8, lo=2000, hi=2000, drop=0,
             cut=0, kv_heads=8, dim=128, page=64, bits=8, layers=1),
        # A step of beam search, 64 requests of 4 beams: most prompts' pages shared by all four.
        dict(name="fork_beams_64x4", op="fork", groups=64, old=4, rows=4, lo=256, hi=4096, drop=16,
             cut=0, kv_heads=8, dim=128, page=64, bits=8, layers=2),
        # A small 4-bit cache after many requests came and went.
        dict(name="compact_4bit_512", op="compact", pages=512, live=0.5, seqs=37, share=0,
             kv_heads=2, dim=64, page=16, bits=4, layers=3),
        # A large one, two thirds in use, prompts' pages shared.
        dict(name="compact_8bit_4096", op="compact", pages=4096, live=0.65, seqs=200, share=8,
             kv_heads=8, dim=128, page=64, bits=8, layers=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append8", "attend8", "attend8", "fork", "compact"])
    page = rng.choice([16, 32, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "append8":
        top = 270336 * 8 * 128 * 2 // (kv_heads * dim * (4 if dtype == "fp32" else 2))
        order = rng.choice(["scattered", "runs"])
        most = min(270336, top) if order == "runs" else min(4096, 270336 // page)
        return dict(op=op, tokens=_log_int(rng, 1, most), kv_heads=kv_heads, dim=dim,
                    page=page, dtype=dtype, order=order)
    if op == "fork":
        groups = _log_int(rng, 1, 100)
        hi = _log_int(rng, 16, max(17, 200000 // groups))
        hi = min(hi, 16000)
        return dict(op=op, groups=groups, old=rng.choice([1, 2, 4]), rows=rng.randint(1, 8),
                    lo=rng.randint(0, hi), hi=hi, drop=rng.choice([0, 4, 16]),
                    cut=rng.choice([0, 0, 40]), kv_heads=kv_heads, dim=dim, page=page,
                    bits=rng.choice([4, 8]), layers=rng.randint(1, 2))
    if op == "compact":
        per = kv_heads * page * dim * 2
        pages = _log_int(rng, 2, max(3, min(20000, 500000000 // per)))
        return dict(op=op, pages=pages, live=rng.uniform(0.05, 0.95), seqs=_log_int(rng, 1, 300),
                    share=rng.choice([0, 3, 8]), kv_heads=kv_heads, dim=dim, page=page,
                    bits=rng.choice([4, 8]), layers=1)
    group = rng.choice([1, 2, 4, 5, 8, 16])
    base = dict(op=op, heads=group * kv_heads, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype)
    kind = rng.choice(["one", "batch", "window", "long", "chunk"])
    if kind == "one":
        n = _log_int(rng, 1, 8192)
        return dict(base, seqs=1, lo=n, hi=n, new_lo=1, new_hi=1)
    if kind == "batch":
        seqs = _log_int(rng, 2, 256)
        hi = _log_int(rng, 16, 8192)
        return dict(base, seqs=seqs, lo=rng.randint(0, hi), hi=hi, new_lo=1, new_hi=1)
    if kind == "window":
        seqs = _log_int(rng, 2, 100)
        hi = _log_int(rng, 16, 16001)
        return dict(base, seqs=seqs, lo=rng.randint(0, hi), hi=hi, new_lo=rng.randint(0, 2),
                    new_hi=rng.randint(2, 8))
    if kind == "long":
        n = _log_int(rng, 8192, 262144)
        return dict(base, seqs=rng.randint(1, 3), lo=n // 2, hi=n, new_lo=1, new_hi=rng.randint(1, 4))
    new = _log_int(rng, 9, 2048)
    hi = max(new, _log_int(rng, 64, 20000))
    return dict(base, seqs=rng.randint(1, 2), lo=new // 2, hi=hi, new_lo=max(1, new // 2), new_hi=new)


# ---------------------------------------------------------- plain helpers ---

def _exponent(top):
    """The least e >= LEAST with top <= 448 2^e."""
    m, x = torch.frexp(top)  # top = m 2^x, 1/2 <= m < 1; 448 = 0.875 * 2^9
    return torch.where(top > 0, x - 9 + (m > 0.875), LEAST).clamp(min=LEAST)


def _code(x):
    """E4M3 bytes of values of magnitude up to 448 (torch rounds to nearest, ties to even)."""
    return x.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _value(codes):
    return codes.contiguous().view(torch.float8_e4m3fn).float()


def _lay(kc, vc):
    """Codes [..., 16, D] of K and V in the order of a group's bytes [..., 16 D] each."""
    D = kc.shape[-1]
    lead = kc.shape[:-2]
    n = len(lead)
    a = kc.reshape(*lead, 16, 4, D // 64, 16).permute(*range(n), n + 2, n, n + 1, n + 3)
    b = vc.reshape(*lead, 2, 4, 2, 8, D // 8).permute(*range(n), n, n + 2, n + 3, n + 1, n + 4)
    return a.reshape(*lead, 16 * D), b.reshape(*lead, 16 * D)


def _unlay(g):
    """The codes [..., 16, D] of K and of V in a group's bytes [..., 32 D + 16]."""
    D = (g.shape[-1] - 16) // 32
    lead = g.shape[:-1]
    n = len(lead)
    a = g[..., :16 * D].reshape(*lead, D // 64, 16, 4, 16).permute(*range(n), n + 1, n + 2, n, n + 3)
    b = g[..., 16 * D:32 * D].reshape(*lead, 2, 2, 8, 4, D // 8)
    b = b.permute(*range(n), n, n + 3, n + 1, n + 2, n + 4)
    return a.reshape(*lead, 16, D), b.reshape(*lead, 16, D)


def _pack(k, v):
    """Groups of 16 tokens: k, v [..., 16, D] -> bytes [..., 32 D + 16]."""
    codes, exps = [], []
    for x in (k, v):
        e = _exponent(x.abs().amax((-2, -1)))
        codes.append(_code(x * torch.exp2(-e.float())[..., None, None]))
        exps.append((e + 127).to(torch.uint8))
    pad = torch.zeros((*k.shape[:-2], 14), dtype=torch.uint8, device=k.device)
    return torch.cat([*_lay(*codes), torch.stack(exps, -1), pad], -1)


def _unpack(g):
    """The inverse: k, v [..., 16, D] fp32."""
    D = (g.shape[-1] - 16) // 32
    e = torch.exp2(g[..., 32 * D:32 * D + 2].float() - 127)
    return [_value(c) * e[..., i, None, None] for i, c in enumerate(_unlay(g))]


# ---------------------------------------------------------------- prepare ---

def _rs_of(case):
    """A case's own random numbers: lengths and the like, so that every seed's outputs have one
    shape and one amount of work."""
    key = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    return np.random.RandomState(zlib.crc32(key.encode()))


def _lengths(case):
    """New and cached tokens of each request; the seed deals them out to the requests."""
    rs = _rs_of(case)
    B = case["seqs"]
    new = rs.randint(case["new_lo"], case["new_hi"] + 1, B)
    kv = rs.randint(case["lo"], case["hi"] + 1, B)
    if case["lo"] > 0:
        kv = np.maximum(kv, new)  # the cache holds the new tokens already
    return new, kv


def _int(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device=DEV)


def prepare(case, seed):
    return {"append8": _prepare_append, "attend8": _prepare_attention, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, seed)


def _filled(pages, heads, groups, D, g):
    """A cache that holds N(0, 1) keys and values."""
    cache = torch.empty((pages, heads, groups, 32 * D + 16), dtype=torch.uint8, device=DEV)
    flat = cache.view(-1, 32 * D + 16)
    chunk = 1 << 17
    for i in range(0, flat.shape[0], chunk):
        n = min(chunk, flat.shape[0] - i)
        k, v = (torch.randn((n, 16, D), device=DEV, generator=g) for _ in range(2))
        flat[i:i + n] = _pack(k, v)
    return cache


def _values(shape, g, dtype):
    """Keys or values: channels of unequal size, a few large ones, some tokens near zero or large."""
    x = torch.randn(shape, device=DEV, generator=g)
    x *= torch.exp2(torch.randn(shape[-2:], device=DEV, generator=g))
    if shape[0]:
        x[torch.rand(shape[0], device=DEV, generator=g) < 0.01] *= 1e-3
        x[torch.rand(shape[0], device=DEV, generator=g) < 0.1] *= 8
    return x.to(dtype)


def _prepare_append(case, seed):
    T, H, D, P = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    rs = np.random.RandomState(seed % (2 ** 31))
    first = _rs_of(case).randint(0, P)
    # k and v are slices of one projection's output, as a model has them
    dtype = DTYPES[case["dtype"]]
    kv = torch.cat([_values((T, H, D), g, dtype), _values((T, H, D), g, dtype)], 1)
    if case["order"] == "runs":  # whole prompts: consecutive slots in pages of any order
        pages = -(-(T + first) // P) + 1
        order = rs.permutation(pages)
        pos = np.arange(T) + first
        slots = order[pos // P] * P + pos % P
        mates = order[0] * P + np.arange(first // 16 * 16, first)
    else:  # one token here and there, each in a block begun earlier
        pages = T + 3
        inside = rs.permutation(_rs_of(case).randint(0, P, T))
        base = rs.permutation(pages)[:T] * P
        slots = base + inside
        mates = np.concatenate([b + np.arange(i // 16 * 16, i) for b, i in zip(base, inside)])
    return dict(case=case, k=kv[:, :H], v=kv[:, H:], slots=_int(slots, torch.int64),
                # the new tokens and those that shared a block with them
                check=_int(np.concatenate([slots, mates]).astype(np.int64), torch.int64),
                cache=_filled(pages, H, P // 16, D, g))


def _deal(pages, need, rs, blocks):
    """Block tables of rows that need so many pages each, pages in any order."""
    ids = rs.permutation(pages)
    table = np.full((len(need), blocks), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, ids[at:]


def _prepare_attention(case, seed):
    rs = np.random.RandomState(seed % (2 ** 31))
    order = rs.permutation(case["seqs"])
    new, kv = (x[order] for x in _lengths(case))
    H, Hk, D, P = (case[x] for x in ("heads", "kv_heads", "dim", "page"))
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = -(-kv // P)
    pages = int(need.sum()) + 2
    table, _ = _deal(pages, need, rs, max(1, int(need.max())))
    cache = _filled(pages, Hk, P // 16, D, g)
    # what lies past a request's end in its last page is another's leftover: any bytes at all
    for b in range(case["seqs"]):
        if kv[b] % P:
            cache[int(table[b, kv[b] // P]), :, (kv[b] % P + 15) // 16:].fill_(255)
    T = int(new.sum())
    q = torch.randn((T, H, D), device=DEV, generator=g) * 1.5
    cu = np.concatenate([[0], np.cumsum(new)])
    return dict(case=case, q=q.to(DTYPES[case["dtype"]]), cache=cache, table=_int(table),
                kv=_int(kv), cu=_int(cu), kv_host=[int(x) for x in kv],
                new_host=[int(x) for x in new], max_new=case["new_hi"])


def _caches(case, pages, g):
    """The layers' caches: pages are moved as they are, so any bytes do."""
    D, H, P = case["dim"], case["kv_heads"], case["page"]
    size = 18 * D if case["bits"] == 4 else 32 * D + 16
    return [torch.randint(0, 256, (pages, H, P // 16, size), dtype=torch.uint8, device=DEV,
                          generator=g) for _ in range(case["layers"])]


def _fork_plan(case):
    """Lengths of the old rows, and of the new ones their parents and what they keep."""
    rs = _rs_of(case)
    G, old, rows = case["groups"], case["old"], case["rows"]
    held = np.repeat(rs.randint(case["lo"], case["hi"] + 1, G), old)
    parents = (np.arange(G) * old)[:, None] + rs.randint(0, old, (G, rows))
    if case["drop"]:  # requests that are over
        parents[rs.randint(0, case["drop"], G) == 0] = -1
    parents = parents.reshape(-1)
    keep = np.where(parents >= 0, held[parents], 0)
    if case["cut"]:  # some go back a few tokens
        keep = np.maximum(0, keep - np.where(rs.rand(len(keep)) < 0.5,
                                             rs.randint(0, case["cut"] + 1, len(keep)), 0))
    return held, parents, keep


def _prepare_fork(case, seed):
    rs = np.random.RandomState(seed % (2 ** 31))
    g = torch.Generator(device=DEV).manual_seed(seed)
    P, G, old = case["page"], case["groups"], case["old"]
    held, parents, keep = _fork_plan(case)
    # the rows of a group share the pages of their prompt, all but their last two
    have = -(-held // P)
    mine = np.minimum(have, 2)
    shared = (have - mine)[::old]
    need = np.concatenate([shared, mine])
    blocks = int(have.max()) + 2
    spare = len(parents) + 5
    pages = int(need.sum()) + spare
    parts, ids = _deal(pages, need, rs, blocks)
    table = np.full((G * old, blocks), -1, np.int64)
    for r in range(G * old):
        n = shared[r // old]
        table[r, :n] = parts[r // old, :n]
        table[r, n:n + mine[r]] = parts[G + r, :mine[r]]
    # the ring of free pages, turned past its end as in a long-running server
    head = int(rs.randint(0, 3 * pages))
    ring = np.full(pages, -1, np.int64)
    ring[(head + np.arange(spare)) % pages] = ids
    return dict(case=case, held=_int(held), table=_int(table), parents=_int(parents),
                keep=_int(keep), ring=_int(ring), span=_int([head, head + spare], torch.int64),
                pages=pages, caches=_caches(case, pages, g))


def _compact_plan(case):
    """Pages of each row, and how many of its first ones it has from the row before."""
    rs = _rs_of(case)
    N, B = case["pages"], case["seqs"]
    live = max(1, min(N - 1, int(N * case["live"])))
    need = rs.multinomial(live, np.ones(B) / B)
    shared = np.zeros(B, np.int64)
    for b in range(1, B):
        if case["share"]:
            shared[b] = rs.randint(0, min(case["share"], need[b - 1]) + 1)
    short = rs.randint(0, case["page"], B)  # tokens missing in the last page
    return need, shared, short


def _prepare_compact(case, seed):
    rs = np.random.RandomState(seed % (2 ** 31))
    g = torch.Generator(device=DEV).manual_seed(seed)
    N, B, P = case["pages"], case["seqs"], case["page"]
    need, shared, short = _compact_plan(case)
    blocks = int((need + shared).max()) + 1
    own_pages, rest = _deal(N, need, rs, blocks)
    table = np.full((B, blocks), -1, np.int64)
    for b in range(B):
        n = shared[b]
        table[b, :n] = own_pages[b - 1, :n]
        table[b, n:n + need[b]] = own_pages[b, :need[b]]
    count = need + shared
    held = np.where(count > 0, count * P - short, 0)
    ring = np.full(N, -1, np.int64)
    ring[:len(rest)] = rest
    return dict(case=case, held=_int(held), table=_int(table), ring=_int(ring), pages=N,
                caches=_caches(case, N, g))


# -------------------------------------------------------------------- run ---

def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import linear_attention_layer_gb300 as kda
        if op == "append8":
            kda.byte_cache_append(state["k"], state["v"], state["slots"], state["cache"])
            return kda.byte_cache_read(state["check"], state["cache"], state["k"].dtype)
        if op == "attend8":
            return kda.byte_cache_attention(
                state["q"], state["cache"], state["table"], state["kv"], state["cu"],
                max_new=state["max_new"], return_lse=True)
        if op == "fork":
            kv, table, copies, span = kda.cache_fork(
                state["held"], state["table"], state["parents"], state["keep"], state["ring"],
                state["span"], page_size=c["page"], num_pages=state["pages"])
            kda.cache_copy(state["caches"], copies)
            return kv, table, copies, span, state["ring"], state["caches"]
        table, copies, span = kda.cache_compact(
            state["held"], state["table"], state["ring"], page_size=c["page"],
            num_pages=state["pages"])
        kda.cache_copy(state["caches"], copies)
        return table, copies, span, state["ring"], state["caches"]
    return {"append8": _plain_append, "attend8": _plain_attention, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


def _plain_append(state):
    c, cache, slots = state["case"], state["cache"], state["slots"]
    D = c["dim"]
    groups = cache.shape[2]
    block, at = slots // 16, slots % 16
    there, which = torch.unique(block, return_inverse=True)
    page, sub = there // groups, there % groups
    bytes_ = cache[page, :, sub]                                   # [blocks, heads, 32 D + 16]
    fresh = torch.zeros(len(there), dtype=torch.bool, device=DEV)
    fresh[which[at == 0]] = True
    codes, exps = list(_unlay(bytes_)), []
    for i, x in enumerate((state["k"], state["v"])):
        e = _exponent(x.float().abs().amax(-1))                    # [tokens, heads]
        top = torch.full((len(there), x.shape[1]), LEAST, dtype=e.dtype, device=DEV)
        top.index_reduce_(0, which, e, "amax")
        old = bytes_[..., 32 * D + i].int() - 127
        new = torch.where(fresh[:, None], top, torch.maximum(top, old))
        # what the block held stands for the same values under the new exponent
        kept = _value(codes[i]) * torch.exp2((old - new).float())[..., None, None]
        codes[i] = torch.where((new > old)[..., None, None], _code(kept), codes[i])
        codes[i][which, :, at] = _code(x.float() * torch.exp2(-new[which].float())[..., None])
        exps.append((new + 127).to(torch.uint8))
    pad = bytes_[..., 32 * D + 2:]
    cache[page, :, sub] = torch.cat([*_lay(*codes), torch.stack(exps, -1), pad], -1)
    block, at = state["check"] // 16, state["check"] % 16
    there, which = torch.unique(block, return_inverse=True)
    k, v = _unpack(cache[there // groups, :, there % groups])
    return k[which, :, at].to(state["k"].dtype), v[which, :, at].to(state["k"].dtype)


def _plain_attention(state):
    c = state["case"]
    H, Hk, D, P = (c[x] for x in ("heads", "kv_heads", "dim", "page"))
    G = H // Hk
    q, cache, table = state["q"], state["cache"], state["table"]
    kv, new, cu = state["kv_host"], state["new_host"], [0]
    for n in new:
        cu.append(cu[-1] + n)
    out = torch.zeros(q.shape, dtype=torch.float32, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float32, device=q.device)
    scale = 1.0 / math.sqrt(D)
    b = 0
    while b < len(kv):  # padded batches of neighbouring requests, as many as fit
        e, L, N = b, 0, 0
        while e < len(kv):
            l2, n2 = max(L, kv[e]), max(N, new[e])
            size = (e + 1 - b) * max(l2 * Hk * D, l2 * n2 * H)
            if e > b and size > (1 << 28):
                break
            e, L, N = e + 1, l2, n2
        if L and N:
            m = e - b
            nb = -(-L // P)
            page = table[b:e, :nb].clamp(min=0).long()
            lens = torch.tensor(kv[b:e], device=q.device)
            news = torch.tensor(new[b:e], device=q.device)
            row = torch.arange(N, device=q.device)
            src = torch.tensor(cu[b:e], device=q.device)[:, None] + row
            live = row < news[:, None]
            qq = q[torch.where(live, src, 0)].float().unflatten(2, (Hk, G))
            key = torch.arange(nb * P, device=q.device)
            inside = key < lens[:, None]
            seen = key <= (lens - news)[:, None, None] + row[:, None]
            seen = seen & inside[:, None] & live[..., None]
            step = max(1, min(Hk, (1 << 30) // max(1, m * N * G * nb * P)))
            for h in range(0, Hk, step):
                k, v = _unpack(cache[page, h:h + step])
                k, v = (torch.where(inside[:, None, :, None],
                                    x.movedim(1, 2).flatten(2, 4), 0.0) for x in (k, v))
                s = torch.einsum("bnhgd,bhld->bhgnl", qq[:, :, h:h + step], k) * scale
                s = s.masked_fill(~seen[:, None, None], -math.inf)
                top = s.amax(-1, keepdim=True).clamp(min=-1e30)
                p = torch.exp(s - top)
                z = p.sum(-1, keepdim=True)
                o = torch.einsum("bhgnl,bhld->bnhgd", p, v)
                o = o / z.clamp(min=1e-30).movedim(3, 1)
                ll = torch.where(z > 0, top + torch.log(z.clamp(min=1e-30)), -math.inf)[..., 0]
                out[src[live], h * G:(h + step) * G] = o.flatten(2, 3)[live]
                lse[src[live], h * G:(h + step) * G] = ll.movedim(3, 1).flatten(2, 3)[live]
        b = e
    return out.to(q.dtype), lse


def _copy_pages(caches, copies):
    """The first tokens of pages, in blocks of 16, from page to page."""
    copies = copies[copies[:, 0] >= 0].long()
    src, dst, n = copies[:, 0], copies[:, 1], copies[:, 2]
    for cache in caches:
        here = torch.arange(cache.shape[2], device=DEV) * 16 < n[:, None]
        cache[dst] = torch.where(here[:, None, :, None], cache[src], cache[dst])


def _plain_fork(state):
    P, N = state["case"]["page"], state["pages"]
    held, parents, keep = state["held"].long(), state["parents"].long(), state["keep"].long()
    old, ring = state["table"], state["ring"].clone()
    head, tail = state["span"][0], state["span"][1]
    cap = ring.numel()
    col = torch.arange(old.shape[1], device=DEV)[None]
    row = torch.arange(parents.numel(), device=DEV)
    keep = torch.where(parents >= 0, keep, 0)
    whole = col < (keep // P)[:, None]
    tails = (keep % P > 0)[:, None] & (col == (keep // P)[:, None])
    table = torch.where(whole | tails, old[parents.clamp(min=0)], -1)
    # an unfinished last page that others hold too: the lowest of the rows that have it unfinished
    # keeps it, unless some row has it whole
    taken = torch.zeros(N + 1, dtype=torch.bool, device=DEV)
    taken[table[whole].long()] = True
    last = torch.where(tails.any(1), torch.where(tails, table, 0).sum(1).long(), N)
    first = torch.full((N + 1,), parents.numel(), dtype=torch.int64, device=DEV)
    first.index_reduce_(0, last, row, "amin")
    move = (last < N) & (taken[last] | (first[last] != row))
    rank = torch.cumsum(move, 0) - move.long()
    page = ring[(head + rank) % cap]
    copies = torch.where(move[:, None], torch.stack([last.int(), page, (keep % P).int()], 1),
                         torch.tensor([-1, -1, 0], dtype=torch.int32, device=DEV))
    table = torch.where(tails & move[:, None], page[:, None], table)
    # pages that were held and are not any more, by their numbers, behind the ring's tail
    before = torch.zeros(N, dtype=torch.bool, device=DEV)
    before[old[col < ((held + P - 1) // P)[:, None]].long()] = True
    after = torch.zeros(N, dtype=torch.bool, device=DEV)
    after[table[whole | tails].long()] = True
    gone = torch.nonzero(before & ~after)[:, 0]
    ring[(tail + torch.arange(gone.numel(), device=DEV)) % cap] = gone.int()
    span = torch.stack([head + move.sum(), tail + gone.numel()])
    _copy_pages(state["caches"], copies)
    return keep.int(), table, copies, span, ring, state["caches"]


def _plain_compact(state):
    P, N = state["case"]["page"], state["pages"]
    held, old, ring = state["held"].long(), state["table"], state["ring"].clone()
    col = torch.arange(old.shape[1], device=DEV)[None]
    mine = col < ((held + P - 1) // P)[:, None]
    live = torch.zeros(N, dtype=torch.bool, device=DEV)
    live[old[mine].long()] = True
    page = torch.arange(N, device=DEV)
    L = live.sum()
    src = torch.nonzero(live & (page >= L))[:, 0]
    dst = torch.nonzero(~live & (page < L))[:, 0]
    to = page.clone()
    to[src] = dst
    table = torch.where(mine, to[old.clamp(min=0).long()].int(), -1)
    copies = torch.tensor([-1, -1, 0], dtype=torch.int32, device=DEV).repeat(N // 2, 1)
    copies[:src.numel()] = torch.stack([src, dst, torch.full_like(src, P)], 1).int()
    free = N - L
    at = torch.arange(ring.numel(), device=DEV)
    ring = torch.where(at < free, (at + L).int(), ring)
    span = torch.stack([torch.zeros_like(free), free])
    _copy_pages(state["caches"], copies)
    return table, copies, span, ring, state["caches"]


# ------------------------------------------------------------------- work ---

def _group_bytes(case):
    return 18 * case["dim"] if case["bits"] == 4 else 32 * case["dim"] + 16


def work(case):
    e = 4 if case.get("dtype") == "fp32" else 2
    if case["op"] == "append8":
        n = 2 * case["tokens"] * case["kv_heads"] * case["dim"]
        return {"bytes": n * (2 * e + 2) + 16 * case["tokens"], "flops": 4 * n}
    if case["op"] == "attend8":
        new, kv = _lengths(case)
        H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
        pairs = sum(int(n) * int(l) - int(n) * (int(n) - 1) // 2 if l >= n
                    else int(l) * (int(l) + 1) // 2 for n, l in zip(new, kv))
        used = sum(int(l) for n, l in zip(new, kv) if n)
        T = int(new.sum())
        return {"bytes": used * Hk * 2 * D + T * H * (2 * D * e + 4), "flops": 4 * D * H * pairs}
    P = case["page"]
    each = case["layers"] * case["kv_heads"] * _group_bytes(case)
    if case["op"] == "fork":
        held, parents, keep = _fork_plan(case)
        # rows of one parent (each has a last page of its own) that are not the first of it
        tail = [(int(p), int(k)) for p, k in zip(parents, keep) if k % P]
        seen, groups = set(), 0
        for p, k in tail:
            if p in seen:
                groups += -(-(k % P) // 16)
            seen.add(p)
        entries = int((-(-held // P)).sum()) + int((-(-keep // P)).sum())
        return {"bytes": 4 * entries + 2 * groups * each, "flops": 0}
    need, shared, _ = _compact_plan(case)
    N, L = case["pages"], int(need.sum())
    moves = L * (N - L) // N  # on average, pages in any order
    return {"bytes": 8 * int((need + shared).sum()) + 4 * (N - L) + 2 * moves * (P // 16) * each,
            "flops": 0}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    if case["op"] == "attend8":
        return _exact_attention(prepare(case, seed))
    if case["op"] == "append8" and case["tokens"] * case["kv_heads"] * case["dim"] <= 1 << 21:
        return _exact_append(prepare(case, seed))
    return None  # whole numbers, or too long to take


def _offsets(D):
    """Byte of K's and of V's code of token i, channel c, in a group [16, D]."""
    i, c = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
    k = c % (D // 4) // 16 * 1024 + i * 64 + c // (D // 4) * 16 + c % 16
    v = 16 * D + (i // 8 * 2 + i % 2) * 4 * D + c // (D // 8) * (D // 2) + i % 8 // 2 * (D // 8) \
        + c % (D // 8)
    return k, v


def _e4m3_table():
    """E4M3 by its definition: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    byte = np.arange(256)
    e, m = byte // 8 % 16, byte % 8
    x = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    x = np.where(byte % 128 == 127, np.nan, x)
    return np.where(byte >= 128, -x, x)


def _nearest(x, scale):
    """The E4M3 value nearest to x / scale, ties to the even code, times scale."""
    grid = _e4m3_table()[:127]
    a = np.abs(x) / scale
    up = np.clip(np.searchsorted(grid, a), 1, 126)
    lo, hi = grid[up - 1], grid[up]
    pick = (hi - a < a - lo) | ((hi - a == a - lo) & (up % 2 == 0))
    return np.where(x < 0, -1.0, 1.0) * np.where(pick, hi, lo) * scale


def _exact_append(st):
    """Block by block, the tokens held before under their old exponent, then the larger one."""
    c = st["case"]
    D, H, P = c["dim"], c["kv_heads"], c["page"]
    table = _e4m3_table()
    cache = st["cache"].cpu().numpy()
    slots = st["slots"].cpu().numpy()
    held = {}  # slot -> values, K and V
    outs = []
    for n, x in enumerate((st["k"], st["v"])):
        x = x.double().cpu().numpy()
        at = _offsets(D)[n]
        values = {}
        start = 0
        while start < len(slots):
            end = start + 1
            while end < len(slots) and slots[end] // 16 == slots[start] // 16:
                end += 1
            page, sub, i = slots[start] // P, slots[start] % P // 16, slots[start] % 16
            raw = cache[page, :, sub]
            old = table[raw[:, at]] * 2.0 ** (raw[:, 32 * D + n].astype(np.float64) - 127)[:, None, None]
            top = np.abs(x[start:end]).max((0, 2))
            with np.errstate(divide="ignore"):
                e = np.maximum(np.ceil(np.log2(top / 448)), LEAST)
            e = np.where(top > 448 * 2.0 ** e, e + 1, e)
            e = np.where((e > LEAST) & (top <= 448 * 2.0 ** (e - 1)), e - 1, e)
            if i:
                e = np.maximum(e, raw[:, 32 * D + n].astype(np.float64) - 127)
            scale = 2.0 ** e[:, None]
            for j in range(i):
                values[slots[start] - i + j] = _nearest(old[:, j], scale)
            for t in range(start, end):
                values[slots[t]] = _nearest(x[t], scale)
            start = end
        held[n] = values
    check = st["check"].cpu().numpy()
    for n in range(2):
        outs.append(torch.from_numpy(np.stack([held[n][s] for s in check])))
    return tuple(outs)


def _exact_attention(st):
    c = st["case"]
    H, Hk, D, P = (c[x] for x in ("heads", "kv_heads", "dim", "page"))
    G = H // Hk
    T = st["q"].shape[0]
    out = torch.zeros((T, H, D), dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    val = torch.from_numpy(_e4m3_table()).to(DEV)
    place = [torch.from_numpy(x).to(DEV).flatten() for x in _offsets(D)]
    at = 0
    for n, l, row in zip(st["new_host"], st["kv_host"], st["table"].cpu().tolist()):
        if n and l:
            pages = torch.tensor(row[:-(-l // P)], device=DEV)
            for h in range(Hk):
                raw = st["cache"][pages, h].flatten(0, 1)       # [groups, 32 D + 16]
                k, v = (
                    (val[raw[:, place[j]].long()].view(-1, 16, D) *
                     torch.exp2(raw[:, 32 * D + j].double() - 127)[:, None, None])
                    .flatten(0, 1)[:l] for j in range(2))
                for r in range(0, n, 512):
                    m = min(512, n - r)
                    q = st["q"][at + r:at + r + m, h * G:(h + 1) * G].double()
                    s = torch.matmul(q, k.T) / math.sqrt(D)  # [m, G, l]
                    last = l - n + r + torch.arange(m, device=DEV)
                    s[(torch.arange(l, device=DEV) > last[:, None])[:, None].expand_as(s)] = -math.inf
                    z = torch.logsumexp(s, -1)
                    p = torch.exp(s - torch.where(z.isinf(), 0.0, z)[..., None])
                    out[at + r:at + r + m, h * G:(h + 1) * G] = torch.matmul(p, v).cpu()
                    lse[at + r:at + r + m, h * G:(h + 1) * G] = z.cpu()
        at += n
    return out, lse
