"""A mixture-of-experts layer with 4-bit weights, run as a serving program would.

    python examples/moe_layer.py [tokens]

Random weights are quantized to 4 bits with a scale and a zero point per group
of 128, laid out once, and one layer is run: a 4-bit projection, the router
(groups, top-k, renormalised weights, and the order of the slots by expert) and
the routed experts.  The router's gradient for a given gradient of its
weights follows.  The result is compared with the same layer computed in
float32 from the dequantized weights.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import binary_packed_weight_gb300 as bpw  # noqa: E402


def quantized(shape, generator, group=128):
    """Random weights as a handle, and as the float32 values the handle stands for."""
    w = torch.randn(shape, generator=generator, device="cuda") * shape[-1] ** -0.5
    lead, K = shape[:-1], shape[-1]
    codes = torch.empty(lead + (K // 2,), dtype=torch.uint8, device="cuda")
    scales = torch.empty(lead + (K // group,), dtype=torch.float16, device="cuda")
    zeros = torch.empty(lead + (K // group,), dtype=torch.uint8, device="cuda")
    bpw.q4_quantize(w, codes, scales, zeros, group=group)
    handle = bpw.q4_upload(codes, scales, zeros, group=group)
    return handle, bpw.q4_dequant(handle, torch.empty((handle.E, handle.N, K), device="cuda"))


def main(tokens=48, D=1024, F=512, E=16, k=4):
    g = torch.Generator(device="cuda").manual_seed(1)
    proj, proj_w = quantized((D, D), g)
    gate, gate_w = quantized((E, F, D), g)
    up, up_w = quantized((E, F, D), g)
    down, down_w = quantized((E, D, F), g)
    router = torch.randn((E, D), generator=g, device="cuda") * D ** -0.5
    hidden = torch.randn((tokens, D), generator=g, device="cuda", dtype=torch.bfloat16)

    x = bpw.q4_gemm(proj, hidden, torch.empty_like(hidden))
    logits = x.float() @ router.T
    ids = torch.empty((tokens, k), dtype=torch.int32, device="cuda")
    weights = torch.empty((tokens, k), device="cuda")
    offsets = torch.empty((E + 1,), dtype=torch.int32, device="cuda")
    slots = torch.empty((tokens * k,), dtype=torch.int32, device="cuda")
    options = dict(score="sigmoid", renorm=True, scale=2.5)
    bpw.moe_route(logits, ids, weights, offsets, slots, groups=4, top_groups=2, **options)
    out = bpw.moe_experts(gate, up, down, x, ids, weights, offsets, slots, torch.empty_like(x))
    dlogits = bpw.moe_route_backward(logits, ids, torch.ones_like(weights), torch.empty_like(logits), **options)
    bpw.device_status()

    want_x = hidden.float() @ proj_w[0].T
    at = ids.long()
    a = torch.einsum("td,tkfd->tkf", x.float(), gate_w[at])
    u = torch.einsum("td,tkfd->tkf", x.float(), up_w[at])
    y = torch.einsum("tkf,tkdf->tkd", torch.nn.functional.silu(a) * u, down_w[at])
    want = (y * weights.unsqueeze(-1)).sum(1)
    errors = {"projection": ((x.float() - want_x).norm() / want_x.norm()).item(),
              "experts": ((out.float() - want).norm() / want.norm()).item(),
              # equal weights' sum does not change with the logits: renormalised, its gradient vanishes
              "gradient of a constant": dlogits.abs().max().item()}
    per_expert = (offsets[1:] - offsets[:-1]).tolist()
    print(f"{tokens} tokens, {k} of {E} experts; slots per expert {per_expert}")
    for name, err in errors.items():
        print(f"  {name}: {err:.2e}")
    return errors


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 48)
