"""An attention layer of a decoder, as a serving program would run it: 4-bit projections, an 8-bit cache.

    python examples/decode_layer.py [prompt tokens] [decoded tokens]

Two sequences share one pool of blocks.  Their prompts go through the layer at once, then tokens one
by one: a 4-bit projection to queries, keys and values, the keys and values into the cache, attention
over it, and a 4-bit projection back.  The last token's result is compared with the layer in float64 from
the dequantized weights and the cache as it reads back.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import binary_packed_weight_gb300 as bpw  # noqa: E402


def quantized(N, K, generator, group=128):
    """A random weight as a handle, and as the values it stands for."""
    w = torch.randn((N, K), generator=generator, device="cuda") * K ** -0.5
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((N, K // group), dtype=torch.float16, device="cuda")
    bpw.q4_quantize(w, codes, scales, group=group)
    handle = bpw.q4_upload(codes, scales, group=group)
    return handle, bpw.q4_dequant(handle, torch.empty((1, N, K), device="cuda"))[0].double()


def main(prompt=100, decoded=5, hidden=512, heads=2, group=4, dim=64, block=32):
    g = torch.Generator(device="cuda").manual_seed(2)
    wide = heads * group
    qkv_w, _ = quantized((wide + 2 * heads) * dim, hidden, g)
    out_w, out_values = quantized(hidden, wide * dim, g)
    seqs, width = 2, -(-(prompt + decoded) // block)
    cache = bpw.KV8Cache(torch.zeros((seqs * width, 2, heads, block, dim), dtype=torch.uint8, device="cuda"),
                         torch.zeros((seqs * width, 2, heads), device="cuda"))
    table = torch.randperm(seqs * width, generator=g, device="cuda").int().view(seqs, width)
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")

    def layer(x, batch, new):
        """x [seqs * new, hidden]: the sequences' next tokens, whose lengths the batch already counts."""
        qkv = bpw.q4_gemm(qkv_w, x, torch.empty((x.shape[0], (wide + 2 * heads) * dim), dtype=x.dtype, device="cuda"))
        qkv = qkv.view(-1, wide + 2 * heads, dim)
        q, k, v = qkv[:, :wide], qkv[:, wide:wide + heads], qkv[:, wide + heads:]
        bpw.kv8_write(cache, batch, k, v)
        a = torch.empty((x.shape[0], wide, dim), dtype=x.dtype, device="cuda")
        bpw.kv8_attention(cache, batch, q, a, max_q=new)
        return q, a, bpw.q4_gemm(out_w, a.view(-1, wide * dim), torch.empty_like(x))

    def batch_of(new):
        offsets = torch.arange(0, seqs * new + 1, new, dtype=torch.int32, device="cuda")
        return bpw.KV8Batch(table, offsets, lens)

    hidden_of = lambda n: torch.randn((seqs * n, hidden), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    step = batch_of(1)
    lens += prompt
    layer(hidden_of(prompt), batch_of(prompt), prompt)
    for _ in range(decoded):
        lens += 1
        q, a, out = layer(hidden_of(1), step, 1)
    bpw.device_status()

    total = prompt + decoded
    k = torch.empty((seqs * total, heads, dim), device="cuda")
    v = torch.empty_like(k)
    bpw.kv8_read(cache, batch_of(total), k, v)
    k, v = (t.view(seqs, total, heads, dim).double() for t in (k, v))
    s = torch.einsum("shgd,sthd->shgt", q.view(seqs, heads, group, dim).double(), k) * dim ** -0.5
    want = torch.einsum("shgt,sthd->shgd", torch.softmax(s, -1), v).reshape(seqs, wide * dim)
    errors = {"attention": ((a.view(seqs, -1).double() - want).norm() / want.norm()).item(),
              "projection": ((out.double() - a.view(seqs, -1).double() @ out_values.T).norm() / out.double().norm()).item()}
    print(f"{seqs} sequences of {prompt} + {decoded} tokens")
    for name, err in errors.items():
        print(f"  {name}: {err:.2e}")
    return errors


if __name__ == "__main__":
    main(*(int(x) for x in sys.argv[1:3]))
