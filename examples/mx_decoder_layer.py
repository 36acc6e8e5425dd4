"""A decoder layer's linears and its query/key path with MX FP4 weights.

Prompts go through W4A4 products (activations quantized to MX FP4 in the call;
once for the two projections that share them), single tokens through W4A16
products (bf16 activations); queries and keys are normalised per head and
rotated in one call, straight from the fused projection's output.  Attention
over whole keys and values is plain torch here; `served` takes the paged 8-bit
cache instead, for prompts and single tokens alike.

    python examples/mx_decoder_layer.py        (needs an MI355X)
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_dequantize_matmul_amd as q4  # noqa: E402


class Layer:
    def __init__(self, hidden=2048, heads=16, kv_heads=8, head=128, ffn=5632, positions=4096, device="cuda:0", seed=0):
        gen = torch.Generator(device).manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.head, self.ffn = hidden, heads, kv_heads, head, ffn

        def weights(n, k):
            return q4.q4_mx_quantize_rows(k ** -0.5 * torch.randn(n, k, generator=gen, device=device))

        self.qkv = weights((heads + 2 * kv_heads) * head, hidden)
        self.out = weights(hidden, heads * head)
        self.gate = weights(ffn, hidden)
        self.up = weights(ffn, hidden)
        self.down = weights(hidden, ffn)
        self.q_gain, self.k_gain = (1 + 0.1 * torch.randn(2, head, generator=gen, device=device)).bfloat16().unbind(0)
        angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, head, 2, device=device, dtype=torch.float64) / head)
        self.cos_sin = torch.cat((angle.cos(), angle.sin()), 1).float()

    def heads_of(self, qkv, positions):
        """The fused projection's rows -> rotated queries, rotated keys, values."""
        T, H, K, D = qkv.shape[0], self.heads, self.kv_heads, self.head
        q = qkv[:, :H * D].view(T, H, D)
        k = qkv[:, H * D:(H + K) * D].view(T, K, D)
        q, k = q4.q4_qk_norm_rope(q, k, self.q_gain, self.k_gain, positions, self.cos_sin)
        return q, k, qkv[:, (H + K) * D:].view(T, K, D)

    def attend(self, q, keys, values, first):
        """Causal attention of queries at positions first .. over one request's cache."""
        T, S, group = q.shape[0], keys.shape[0], self.heads // self.kv_heads
        k = keys.float().repeat_interleave(group, 1).permute(1, 2, 0).contiguous()
        v = values.float().repeat_interleave(group, 1).transpose(0, 1).contiguous()
        score = torch.matmul(q.float().transpose(0, 1).contiguous(), k) * self.head ** -0.5
        ahead = torch.arange(S, device=q.device) > first + torch.arange(T, device=q.device)[:, None]
        p = torch.softmax(score.masked_fill(ahead, float("-inf")), 2)
        return torch.matmul(p, v).transpose(0, 1).reshape(T, -1).bfloat16()

    def prompt(self, x, lengths):
        """bf16 rows of several prompts, one after the other -> (rows, caches)."""
        at = torch.cat([torch.arange(n, device=x.device) for n in lengths])
        q, k, v = self.heads_of(q4.q4_linear_w4a4_mx_dynamic(x, *self.qkv), at)
        caches = list(zip(k.split(lengths), v.split(lengths)))
        a = torch.cat([self.attend(qi, *c, 0) for qi, c in zip(q.split(lengths), caches)])
        x = x + q4.q4_linear_w4a4_mx_dynamic(a, *self.out)
        xq = q4.q4_mx_quantize_rows(x)          # one set of codes for both projections
        h = torch.nn.functional.silu(q4.q4_linear_w4a4_mx(*xq, *self.gate)) * q4.q4_linear_w4a4_mx(*xq, *self.up)
        return x + q4.q4_linear_w4a4_mx_dynamic(h, *self.down), caches

    def token(self, x, caches):
        """One bf16 row a request -> (rows, caches with the token)."""
        at = torch.tensor([k.shape[0] for k, _ in caches], device=x.device)
        q, k, v = self.heads_of(q4.q4_linear_w4a16_mx(x, *self.qkv), at)
        caches = [(torch.cat((ck, k[i:i + 1])), torch.cat((cv, v[i:i + 1]))) for i, (ck, cv) in enumerate(caches)]
        a = torch.cat([self.attend(q[i:i + 1], *c, c[0].shape[0] - 1) for i, c in enumerate(caches)])
        x = x + q4.q4_linear_w4a16_mx(a, *self.out)
        h = torch.nn.functional.silu(q4.q4_linear_w4a16_mx(x, *self.gate)) * q4.q4_linear_w4a16_mx(x, *self.up)
        return x + q4.q4_linear_w4a16_mx(h, *self.down), caches

    def served(self, x, cache, pages, starts, lengths):
        """bf16 rows of the requests' new tokens, one request after the other -> rows.
        lengths int32 [N] count the new tokens, starts int32 [N + 1] are where a request's rows begin."""
        T, H, K, D = x.shape[0], self.heads, self.kv_heads, self.head
        linear = q4.q4_linear_w4a16_mx if T == pages.shape[0] else q4.q4_linear_w4a4_mx_dynamic
        qkv = linear(x, *self.qkv).view(T, H + 2 * K, D)
        q = q4.q8_kv_append(cache, pages, starts, lengths, qkv[:, H:H + K], qkv[:, H + K:], qkv[:, :H], self.cos_sin,
                            self.k_gain, self.q_gain, eps=1e-6)
        x = x + linear(q4.q8_attention(q, cache, pages, starts, lengths).view(T, H * D), *self.out)
        h = torch.nn.functional.silu(linear(x, *self.gate)) * linear(x, *self.up)
        return x + linear(h, *self.down)


def main():
    layer, lengths = Layer(), [700, 37, 1, 290]
    gen = torch.Generator("cuda:0").manual_seed(1)
    x = torch.randn(sum(lengths), layer.hidden, generator=gen, device="cuda:0").bfloat16()
    for run in ("first", "second"):
        torch.cuda.synchronize()
        t = time.perf_counter()
        y, caches = layer.prompt(x, lengths)
        torch.cuda.synchronize()
        t1 = time.perf_counter()
        z = torch.randn(len(lengths), layer.hidden, generator=gen, device="cuda:0").bfloat16()
        for _ in range(8):
            z, caches = layer.token(z, caches)
        torch.cuda.synchronize()
        print(f"{run} run: {x.shape[0]} prompt rows {1e3 * (t1 - t):.2f} ms, 8 tokens of {len(lengths)} requests "
              f"{1e3 * (time.perf_counter() - t1):.2f} ms")
    assert torch.isfinite(y).all() and torch.isfinite(z).all()

    width = -(-(max(lengths) + 16) // 64)
    pages = torch.arange(len(lengths) * width, dtype=torch.int32, device="cuda:0").view(-1, width)
    cache = q4.q8_kv_cache(pages.numel(), layer.kv_heads, 64, layer.head)
    starts = torch.tensor([0, 700, 737, 738, 1028], dtype=torch.int32, device="cuda:0")
    ones = torch.arange(len(lengths) + 1, dtype=torch.int32, device="cuda:0")
    for run in ("first", "second"):
        have = torch.tensor(lengths, dtype=torch.int32, device="cuda:0")
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = layer.served(x, cache, pages, starts, have)
        torch.cuda.synchronize()
        t1 = time.perf_counter()
        z = torch.randn(len(lengths), layer.hidden, generator=gen, device="cuda:0").bfloat16()
        for _ in range(8):
            have += 1
            z = layer.served(z, cache, pages, ones, have)
        torch.cuda.synchronize()
        print(f"{run} run, 8-bit cache: {x.shape[0]} prompt rows {1e3 * (t1 - t):.2f} ms, 8 tokens of {len(lengths)} "
              f"requests {1e3 * (time.perf_counter() - t1):.2f} ms")
    assert torch.isfinite(y).all() and torch.isfinite(z).all()


if __name__ == "__main__":
    main()
