"""A decoder layer on 4-bit weights, served from a paged cache.

    python examples/decoder_layer.py [--steps 50] [--users 16] [--prompt 700] [--cache-bits 16]

Each user's prompt runs through the layer in one call (chunks of different lengths side by side),
then all users decode a token at a time, the step captured in a graph.  Projections are
`linear` calls with their epilogues, positions and the cache `kv_append`, attention
`paged_attention` (with `--cache-bits 4` `kv4_append` and `kv4_attention`); only the norm is torch's.  Weights are random, quantised by `quantize`.
The last step's outputs are compared with the same layer in fp32 on the dequantised weights, with a cache
of 4 bits on the keys and values that it stands for.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_quantized_qmm_amd as qmm  # noqa: E402

BITS, G = 4, 128


class Weight:
    """A K x N matrix as 4-bit codes with one scale and zero-point for each group of 128 rows."""

    def __init__(self, K, N, gen):
        codes, self.s, self.z = qmm.quantize((torch.randn(K, N, generator=gen, device="cuda") * K ** -0.5).half(), BITS, G)
        self.wq = qmm.pack(codes, BITS)
        self.codes = codes

    def __call__(self, x, **epilogue):
        return qmm.linear(x, self.wq, self.s, self.z, BITS, G, **epilogue)

    def dense(self):
        s, z = (t.float().repeat_interleave(G, 1).t() for t in (self.s, self.z))
        return (self.codes.float() - z) * s


def norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).half()


class Layer:
    def __init__(self, hidden, heads, kv_heads, head_dim, inner, gen):
        self.Hq, self.Hkv, self.D = heads, kv_heads, head_dim
        self.qkv = Weight(hidden, (heads + 2 * kv_heads) * head_dim, gen)
        self.o = Weight(heads * head_dim, hidden, gen)
        self.gate, self.up, self.down = Weight(hidden, inner, gen), Weight(hidden, inner, gen), Weight(inner, hidden, gen)

    def split(self, qkv):
        cut = (self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D)
        return (t.unflatten(1, (-1, self.D)) for t in qkv.split(cut, 1))

    def __call__(self, x, cache, slots, positions, rope, table, cu_q, kv_lens, max_q, max_kv):
        q, k, v = self.split(self.qkv(norm(x)))
        if isinstance(cache, qmm.KV4Cache):
            q = qmm.kv4_append(q, k, v, cache, slots, positions, rope)
            a = qmm.kv4_attention(q, cache, table, cu_q, kv_lens, max_q, max_kv)
        else:
            q = qmm.kv_append(q, k, v, cache[0], cache[1], slots, positions, rope)
            a = qmm.paged_attention(q, cache[0], cache[1], table, cu_q, kv_lens, max_q, max_kv)
        x = self.o(a.flatten(1), residual=x)
        h = norm(x)
        return self.down(self.gate(h, act="silu", mul=self.up(h)), residual=x)

    def reference(self, x, rope, cached=None):
        """One user's whole sequence in fp32; `cached`: keys and values to take instead of its own."""
        L, rot = x.shape[0], rope.shape[1]
        x = x.float()
        q, k, v = self.split(norm(x).float() @ self.qkv.dense())
        c, s = rope[:L, None, :rot // 2], rope[:L, None, rot // 2:]
        q, k = (torch.cat((t[..., :rot // 2] * c - t[..., rot // 2:] * s, t[..., rot // 2:] * c + t[..., :rot // 2] * s), -1) for t in (q, k))
        k, v = (t.float().repeat_interleave(self.Hq // self.Hkv, 1) for t in cached or (k, v))
        score = torch.stack([q[:, h] @ k[:, h].t() for h in range(self.Hq)]) * self.D ** -0.5
        p = torch.softmax(score.masked_fill(torch.ones(L, L, device=x.device, dtype=torch.bool).triu(1), -torch.inf), -1)
        x = x + torch.stack([p[h] @ v[:, h] for h in range(self.Hq)], 1).flatten(1) @ self.o.dense()
        h = norm(x).float()
        g = h @ self.gate.dense()
        return x + (g * torch.sigmoid(g) * (h @ self.up.dense())) @ self.down.dense()


def run(hidden=4096, heads=32, kv_heads=8, head_dim=128, inner=14336, users=16, prompt=700, steps=50, page=16, seed=0, cache_bits=16):
    """Prompts, then `steps` decode steps; returns (us a decode step, relative error of a user's last output)."""
    dev, gen = "cuda", torch.Generator(device="cuda")
    gen.manual_seed(seed)
    layer = Layer(hidden, heads, kv_heads, head_dim, inner, gen)
    lens = [max(1, prompt - 37 * u % prompt) for u in range(users)]
    most = max(lens) + steps
    width = -(-most // page)
    if cache_bits == 4:
        cache = qmm.kv4_cache(users * width, kv_heads, page, head_dim)
    else:
        cache = tuple(torch.zeros(users * width, kv_heads, page, head_dim, device=dev, dtype=torch.float16) for _ in range(2))
    table = torch.randperm(users * width, generator=gen, device=dev).to(torch.int32).view(users, width)
    angle = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(head_dim // 2, device=dev, dtype=torch.float64) * 2 / head_dim)
    rope = torch.cat((angle.cos(), angle.sin()), 1).float()
    tokens = [torch.randn(n + steps, hidden, generator=gen, device=dev).half() for n in lens]     # what the layer is given

    def slots_of(user, pos):
        return table[user, pos // page].long() * page + pos % page

    user = torch.cat([torch.full((n,), u, device=dev) for u, n in enumerate(lens)])
    pos = torch.cat([torch.arange(n, device=dev) for n in lens])
    cu = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
    kv = torch.tensor(lens, device=dev, dtype=torch.int32)
    layer(torch.cat([t[:n] for t, n in zip(tokens, lens)]), cache, slots_of(user, pos), pos.to(torch.int32), rope, table, cu, kv, max(lens), max(lens))

    # one decode step on buffers that the graph reads
    x = torch.empty(users, hidden, device=dev, dtype=torch.float16)
    one, every = torch.arange(users + 1, device=dev, dtype=torch.int32), torch.arange(users, device=dev)
    positions, slots = torch.empty(users, device=dev, dtype=torch.int32), torch.empty(users, device=dev, dtype=torch.int64)

    def feed(step):
        x.copy_(torch.stack([t[n + step] for t, n in zip(tokens, lens)]))
        positions.copy_(kv)
        slots.copy_(slots_of(every, positions.long()))
        kv.add_(1)

    def step():
        return layer(x, cache, slots, positions, rope, table, one, kv, 1, most)

    feed(0)
    step()                                    # (writes the cache's same places as its replay)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    spent = 0.0
    for i in range(1, steps):
        feed(i)
        torch.cuda.synchronize()
        t = time.perf_counter()
        graph.replay()
        torch.cuda.synchronize()
        spent += time.perf_counter() - t
    u = users // 2
    held = qmm.kv4_read(cache, slots_of(u, torch.arange(lens[u] + steps, device=dev))) if cache_bits == 4 else None
    want = layer.reference(tokens[u], rope, held)[-1]
    error = float((out[u].float() - want).norm() / want.norm())
    return spent / max(1, steps - 1) * 1e6, error


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, value in (("steps", 50), ("users", 16), ("prompt", 700)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--cache-bits", type=int, choices=(4, 16), default=16)
    a = ap.parse_args()
    us, error = run(users=a.users, prompt=a.prompt, steps=a.steps, cache_bits=a.cache_bits)
    print(f"decode step of one layer, {a.users} users, prompts up to {a.prompt}, cache of {a.cache_bits} bits: {us:.1f} us; relative error of the last output {error:.1e}")
