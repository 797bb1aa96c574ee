"""Serving a small hybrid model: three KDA layers, then one layer of grouped-query attention.

A KDA layer's memory of a request is a state of fixed size (fp32, updated in place); the
attention layer's is the 4-bit paged cache.  One step of the server, whatever each request
brings -- a prompt, a chunk of one, one token, a window of drafts -- is

    cache_tables      pages for the new tokens, given back for rejected ones
    per block         chunk_fwd (or decode_step) three times,
                      cache_append + cache_attention once

with random weights: ``python examples/hybrid_serving.py`` runs a prompt phase, decode
steps and a window of drafts that is partly rejected, and prints what the cache holds.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_layer_gb300 as kda  # noqa: E402


class HybridModel:
    """Random weights of ``blocks`` blocks of three KDA layers and one attention layer."""

    def __init__(self, width=512, kda_heads=4, heads=8, kv_heads=2, blocks=1, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, m):
            w = torch.randn((n, m), device=device, generator=g) * n ** -0.5
            return w.to(torch.bfloat16)

        self.kda_heads, self.heads, self.kv_heads, self.blocks = kda_heads, heads, kv_heads, blocks
        self.dim, self.device = 128, device
        D = self.dim
        self.kda = [[dict(qkvz=weight(width, 4 * kda_heads * D), beta=weight(width, kda_heads),
                          out=weight(kda_heads * D, width)) for _ in range(3)]
                    for _ in range(blocks)]
        self.attention = [dict(qkv=weight(width, (heads + 2 * kv_heads) * D),
                               out=weight(heads * D, width)) for _ in range(blocks)]


def _norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Server:
    """Up to ``slots`` requests at a time; one ``step`` feeds each of them some tokens."""

    def __init__(self, model, slots, pages, page_size=64, max_blocks=64):
        m, dev = model, model.device
        self.model, self.page_size = model, page_size
        self.states = [[torch.zeros((slots, m.kda_heads, m.dim, m.dim), device=dev)
                        for _ in range(3)] for _ in range(m.blocks)]
        self.caches = [kda.cache_empty(pages, page_size, m.kv_heads, m.dim, dev)
                       for _ in range(m.blocks)]
        self.table = torch.full((slots, max_blocks), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(pages, dtype=torch.int32, device=dev)
        self.free_range = torch.tensor([0, pages], device=dev)
        self.held = torch.zeros(slots, dtype=torch.int32, device=dev)

    def step(self, x, new, keep=None):
        """x [T, width]: the new tokens of the requests one after another, ``new`` of each
        (-1: the request is over, its slot free for another).  ``keep``: tokens of each that stay (default: all; fewer
        after drafts were rejected -- the KDA states are then the caller's to restore).
        Returns the outputs [T, width]."""
        m = self.model
        count = [max(n, 0) for n in new]
        new_lens = torch.tensor(new, dtype=torch.int32, device=x.device)
        seq = self.held if keep is None else torch.tensor(keep, dtype=torch.int32, device=x.device)
        lens, cu, slots, self.free_range = kda.cache_tables(
            self.held, seq, new_lens, self.table, self.free, self.free_range,
            page_size=self.page_size, max_tokens=x.shape[0])
        self.held = lens
        offsets = [0]
        for n in count:
            offsets.append(offsets[-1] + n)
        over = [b for b, n in enumerate(new) if n < 0]
        if over:  # pages go back in cache_tables; a state stays until it is cleared
            for states in self.states:
                for state in states:
                    state[over] = 0
        for layers, states, att, cache in zip(m.kda, self.states, m.attention, self.caches):
            for w, state in zip(layers, states):
                x = x + self._kda(w, state, _norm(x), cu, offsets)
            x = x + self._attention(att, cache, _norm(x), slots, lens, cu, max(count + [1]))
        return x

    def _kda(self, w, state, x, cu, offsets):
        m, T = self.model, x.shape[0]
        q, k, v, z = (x @ w["qkvz"]).view(T, 4, m.kda_heads, m.dim).unbind(1)
        beta = torch.sigmoid((x @ w["beta"]).float())
        q, k, v, z = q.contiguous(), k.contiguous(), v.contiguous(), z.float().contiguous()
        if T == len(offsets) - 1 and offsets == list(range(T + 1)):  # one token each
            o = kda.decode_step(q, k, v, z, beta, state)
        else:
            o, _ = kda.chunk_fwd(q, k, v, z, beta, cu, state, final_state=state,
                                 cu_seqlens_host=offsets)
        return o.reshape(T, -1) @ w["out"]

    def _attention(self, w, cache, x, slots, lens, cu, longest):
        m, T = self.model, x.shape[0]
        qkv = (x @ w["qkv"]).view(T, m.heads + 2 * m.kv_heads, m.dim)
        q, k, v = qkv.split([m.heads, m.kv_heads, m.kv_heads], dim=1)  # views: strides, no copies
        kda.cache_append(k, v, slots, cache)
        o = kda.cache_attention(q, cache, self.table, lens, cu, max_new=longest)
        return o.reshape(T, -1) @ w["out"]

    def snapshot(self):
        return [[s.clone() for s in states] for states in self.states]

    def restore(self, snap):
        for states, kept in zip(self.states, snap):
            for s, k in zip(states, kept):
                s.copy_(k)


def main():
    torch.manual_seed(0)
    model = HybridModel(blocks=2)
    server = Server(model, slots=4, pages=64)

    def tokens(n):
        return torch.randn((n, 512), device="cuda").to(torch.bfloat16)

    prompts = [300, 17, 1, 130]
    server.step(tokens(sum(prompts)), prompts)
    for _ in range(8):
        server.step(tokens(4), [1, 1, 1, 1])
    before, lens = server.snapshot(), server.held.tolist()
    server.step(tokens(12), [3, 3, 3, 3])  # drafts
    server.restore(before)  # request b keeps accepted[b] of its three: replay those
    accepted = [3, 0, 1, 2]
    server.step(tokens(sum(accepted)), accepted, keep=lens)
    server.step(tokens(3), [1, 1, -1, 1])  # the third request is over
    head, tail = server.free_range.tolist()
    error = kda.get_device_error()
    print(f"lengths {server.held.tolist()}, free pages {tail - head} of 64, "
          f"cache {sum(c.numel() for c in server.caches) / 2 ** 20:.1f} MiB, "
          f"device error {error}")
    return error


if __name__ == "__main__":
    sys.exit(main())
