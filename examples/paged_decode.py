"""One attention block of a decode layer over a paged cache, served in steps.

    python examples/paged_decode.py

A step takes up to eight tokens of any requests: chunks of new prompts, single
tokens, or both.  Five launches run it: the qkv product of all columns, the block
tables and slot maps from the requests' lengths, rotary positions with the write
into the cache, attention over the cache, and the output product with the residual.
The same buffers serve every step, so a step is captured into a graph once and
replayed for whatever lengths the buffers then hold; tokens past a step's own are
padding, without a place in the cache."""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from decode_gemv_elementwise_amd import binding, paged, synth  # noqa: E402

COLUMNS = 8  # tokens of a step: what one product call takes


class Block:
    """Weights and buffers; ``hidden`` values a token, heads of ``dim`` values."""

    def __init__(self, hidden=4096, heads=32, kv_heads=8, dim=128, page=16, pages=256, requests=4, longest=1024, window=0,
                 sinks=0, seed=0):
        rng = np.random.default_rng(seed)
        self.hidden, self.heads, self.kv_heads, self.dim, self.page = hidden, heads, kv_heads, dim, page
        self.window, self.sinks, self.longest = window, sinks, longest
        self.rows = (heads + 2 * kv_heads) * dim
        self.w_qkv = synth.random_weights(rng, "bf16", self.rows, hidden)
        self.w_out = synth.random_weights(rng, "bf16", hidden, heads * dim)
        dev = torch.device("cuda")
        self.qkv_data, self.out_data = (torch.from_numpy(w.data).to(dev) for w in (self.w_qkv, self.w_out))
        ints = lambda *n: torch.zeros(n, dtype=torch.int32, device=dev)  # noqa: E731
        floats = lambda *n: torch.zeros(n, device=dev)  # noqa: E731
        self.x, self.qkv, self.mixed, self.y = (floats(COLUMNS, hidden), floats(COLUMNS, self.rows),
                                                floats(COLUMNS, heads, dim), floats(COLUMNS, hidden))
        self.q = torch.zeros(COLUMNS, heads, dim, dtype=torch.bfloat16, device=dev)
        self.k_cache, self.v_cache = (torch.zeros(pages, page, kv_heads, dim, dtype=torch.bfloat16, device=dev) for _ in "kv")
        self.inv_freq = (10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64) / (dim // 2))).float().to(dev)
        self.cached, self.fresh = ints(requests), ints(requests)
        self.table = torch.full((requests, -(-longest // page)), -1, dtype=torch.int32, device=dev)
        self.query_start, self.kv_len, self.used = ints(requests + 1), ints(requests), ints(1)
        self.request, self.positions, self.slots = ints(COLUMNS), ints(COLUMNS), ints(COLUMNS)
        self.pool = list(range(pages))  # pages that nobody holds
        self.free = ints(COLUMNS)       # those that the step may take: one a token at most
        self.workspace = paged.attn_workspace(dim)
        self.lengths = [0] * requests
        self.graph = None

    def launches(self):
        t, d = COLUMNS, self.dim
        binding.gemv_fused_ncols(self.qkv_data, "bf16", self.rows, self.hidden, t, self.x, "none", dst=self.qkv)
        paged.gemv_paged_slots(self.cached, self.fresh, self.free, self.page, self.table, self.query_start, self.kv_len,
                               self.request, self.positions, self.slots, self.used)
        q, k, v = self.qkv.split([self.heads * d, self.kv_heads * d, self.kv_heads * d], 1)
        paged.gemv_paged_append(q.unflatten(1, (-1, d)), k.unflatten(1, (-1, d)), v.unflatten(1, (-1, d)), self.positions,
                                self.inv_freq, self.slots, self.q, self.k_cache, self.v_cache)
        paged.gemv_paged_attn(self.q, self.k_cache, self.v_cache, self.table, self.query_start, self.kv_len, d ** -0.5,
                              self.mixed, self.workspace, window=self.window, sinks=self.sinks)
        binding.gemv_fused_ncols(self.out_data, "bf16", self.hidden, self.heads * d, t, self.mixed, "add",
                                 add_operand=self.x, dst=self.y)

    def step(self, x, fresh, graph=True):
        """x: [tokens, hidden], the requests' new tokens in their order; fresh: how many each has.  Returns [tokens, hidden].
        A step that needs more pages than are free, or takes a request past ``longest``, is refused before it takes any."""
        n = sum(fresh)
        assert x.shape == (n, self.hidden) and 0 < n <= COLUMNS and len(fresh) == len(self.lengths)
        need = sum(-(-(c + f) // self.page) - -(-c // self.page) for c, f in zip(self.lengths, fresh))
        if max(c + f for c, f in zip(self.lengths, fresh)) > self.longest:
            raise ValueError(f"a request would be longer than {self.longest} tokens")
        if need > len(self.pool):
            raise ValueError(f"{need} pages needed, {len(self.pool)} free")
        taken, self.pool = self.pool[:need], self.pool[need:]
        self.x[:n].copy_(x)
        self.cached.copy_(torch.tensor(self.lengths, dtype=torch.int32))
        self.fresh.copy_(torch.tensor(fresh, dtype=torch.int32))
        self.free.copy_(torch.tensor(taken + [-1] * (COLUMNS - need), dtype=torch.int32))
        if not graph:
            self.launches()
        else:
            if self.graph is None:
                saved = [t.clone() for t in (self.table, self.k_cache, self.v_cache)]
                self.launches()  # once outside: the library loads its code
                torch.cuda.synchronize()
                for t, s in zip((self.table, self.k_cache, self.v_cache), saved):
                    t.copy_(s)
                self.graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(self.graph):
                    self.launches()
            self.graph.replay()
        self.lengths = [c + f for c, f in zip(self.lengths, fresh)]
        return self.y[:n].clone()

    def release(self, request):
        """Gives a finished request's pages back."""
        held = self.table[request].tolist()[:-(-self.lengths[request] // self.page)]
        self.pool += held
        self.table[request] = -1
        self.lengths[request] = 0


def main():
    block = Block()
    g = torch.Generator(device="cuda").manual_seed(0)
    tokens = lambda n: torch.randn(n, block.hidden, generator=g, device="cuda")  # noqa: E731
    for fresh in ([8, 0, 0, 0], [1, 7, 0, 0], [1, 1, 6, 0], [1, 1, 1, 5]):
        block.step(tokens(sum(fresh)), fresh)
    torch.cuda.synchronize()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in "ab")
    start.record()
    for _ in range(100):
        block.graph.replay()  # the last step again and again: launches alone
    end.record()
    torch.cuda.synchronize()
    print(f"a step of four requests: {start.elapsed_time(end) * 10:.1f} us on the GPU, {len(block.pool)} pages free")
    y = block.step(tokens(4), [1, 1, 1, 1])
    print(f"lengths {block.lengths}, result {tuple(y.shape)}, mean square {float(y.square().mean()):.3f}")
    block.release(0)
    print(f"after the first request's end: {len(block.pool)} pages free")


if __name__ == "__main__":
    main()
