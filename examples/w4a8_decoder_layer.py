"""A decoder layer as it is served: int4 weights, int8 activations, an 8-bit cache.

Prompts and single tokens take the same steps: rows are normalised straight to
int8 codes, the fused projection, keys and values into the paged cache (with the
heads' norms and the rotation of queries and keys), attention over the cache, the
output projection, and the gated feed forward network behind a second norm, which
adds the residual on its way.  Which rows belong to which request is on
the device (starts, lengths, pages), so a step of single tokens is captured into
a graph once and replayed for every further token.

    python examples/w4a8_decoder_layer.py        (needs an MI355X)
"""
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_dequantize_matmul_amd as q4  # noqa: E402


class Layer:
    def __init__(self, hidden=2048, heads=16, kv_heads=8, head=128, ffn=5632, positions=4096, device="cuda:0", seed=0):
        rng = np.random.default_rng(seed)
        self.hidden, self.heads, self.kv_heads, self.head, self.ffn = hidden, heads, kv_heads, head, ffn

        def weights(n, k):
            packed, scales = q4.q4_quantize_matrix(k ** -0.5 * rng.standard_normal((n, k), dtype=np.float32))
            return torch.from_numpy(packed).to(device), torch.from_numpy(scales).to(device)

        def gain(n):
            return torch.from_numpy(1 + 0.1 * rng.standard_normal(n, dtype=np.float32)).to(device)

        self.qkv = weights((heads + 2 * kv_heads) * head, hidden)
        self.out = weights(hidden, heads * head)
        self.gate_up = weights(2 * ffn, hidden)
        self.down = weights(hidden, ffn)
        self.gain_in, self.gain_ffn, self.gain_q, self.gain_k = gain(hidden), gain(hidden), gain(head), gain(head)
        angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, head, 2, device=device, dtype=torch.float64) / head)
        self.cos_sin = torch.cat((angle.cos(), angle.sin()), 1).float()

    def step(self, x, cache, pages, starts, lengths):
        """f32 rows of the requests' new tokens, one request after the other -> rows.
        lengths count the new tokens; starts are where each request's rows begin."""
        H, K, D = self.heads, self.kv_heads, self.head
        T = x.shape[0]
        codes, scales, _ = q4.q8_rmsnorm_rows(x, self.gain_in)
        qkv = q4.q4_linear_w4a8(codes, scales, *self.qkv).view(T, H + 2 * K, D)
        q = q4.q8_kv_append(cache, pages, starts, lengths, qkv[:, H:H + K], qkv[:, H + K:], qkv[:, :H], self.cos_sin,
                            self.gain_k, self.gain_q, eps=1e-6)
        a = q4.q8_attention(q, cache, pages, starts, lengths).view(T, H * D)
        a = q4.q4_linear_w4a8_dynamic(a, *self.out)
        codes, scales, x = q4.q8_rmsnorm_rows(a, self.gain_ffn, x, total=a)
        gate, up = q4.q4_linear_w4a8(codes, scales, *self.gate_up).chunk(2, 1)
        return x + q4.q4_linear_w4a8_dynamic(torch.nn.functional.silu(gate) * up, *self.down)


def tables(lengths, more, page, device="cuda:0"):
    """A cache's pages, in any order, for requests of these lengths and `more` tokens each -> (page count, table)."""
    need = [-(-(n + more) // page) for n in lengths]
    order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(2)).int()
    table = torch.zeros(len(lengths), max(need), dtype=torch.int32)
    for row, own in zip(table, order.split(need)):
        row[:len(own)] = own
    return sum(need), table.to(device)


def main():
    layer, prompts, tokens = Layer(), [700, 37, 1, 290], 8
    gen = torch.Generator("cuda:0").manual_seed(1)
    count, pages = tables(prompts, 4 * tokens, 64)
    cache = q4.q8_kv_cache(count, layer.kv_heads, 64, layer.head)
    starts = torch.tensor(np.cumsum([0] + prompts), dtype=torch.int32, device="cuda:0")
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda:0")
    x = torch.randn(sum(prompts), layer.hidden, generator=gen, device="cuda:0")
    for run in ("first", "second"):
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = layer.step(x, cache, pages, starts, lengths)
        torch.cuda.synchronize()
        print(f"{run} run: {x.shape[0]} prompt rows {1e3 * (time.perf_counter() - t):.2f} ms")

    ones = torch.arange(len(prompts) + 1, dtype=torch.int32, device="cuda:0")
    z = torch.randn(len(prompts), layer.hidden, generator=gen, device="cuda:0")

    def token():
        lengths.add_(1)
        z.copy_(layer.step(z, cache, pages, ones, lengths))

    token()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token()
    for name, run in (("call by call", token), ("replayed", graph.replay)):
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(tokens):
            run()
        torch.cuda.synchronize()
        print(f"{tokens} tokens of {len(prompts)} requests {name}: {1e3 * (time.perf_counter() - t):.2f} ms")
    assert torch.isfinite(y).all() and torch.isfinite(z).all()


if __name__ == "__main__":
    main()
