"""A routed layer in graphs, on several streams, and what its calls keep of the device's memory."""
import os
import subprocess
import sys

import numpy as np
import pytest

from test_gpu_moe_ranges import layer

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def moe_call(lib, rng, T, E=8, k=2, D=256, F=128, dtype="bfloat16"):
    """A routed layer and what it needs: (call(out), out, inputs that may be overwritten)."""
    import torch
    _, handles = layer(lib, rng, E, D, F)
    l = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)).cuda()
    x = torch.from_numpy(rng.normal(size=(T, D))).to(getattr(torch, dtype)).cuda()
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    off, slots = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T * k, dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)

    def call():
        lib.moe_route(l, ids, w, off, slots)
        lib.moe_experts(*handles, x, ids, w, off, slots, out)
        return out
    return call, out, l, x


@pytest.mark.parametrize("T,dtype", [(1, "float32"), (16, "bfloat16"), (40, "float16"), (1500, "bfloat16")])
def test_layer_in_a_graph(lib, T, dtype):
    """Routing, plan, scratch and products captured once and replayed on other inputs."""
    import torch
    call, out, l, x = moe_call(lib, np.random.default_rng(80), T, dtype=dtype)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        l.copy_(torch.randn_like(l))
        x.copy_(torch.randn_like(x))
        want = call().clone()
        out.fill_(7.0)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    lib.device_status()


FIRST = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import numpy as np, torch
import binary_packed_weight_gb300 as lib
from test_gpu_moe_sharing import moe_call
call, out, l, x = moe_call(lib, np.random.default_rng(81), {T})
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
got = out.clone()
assert torch.equal(call(), got)
lib.device_status()
print("as captured")
"""


@pytest.mark.parametrize("T", [3, 1500])
def test_first_call_of_a_process_may_be_captured(lib, T):
    """What the library keeps (its pool, limits of the kernels) is made by the first call, which may be a capture."""
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, T=T)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as captured" in r.stdout, r.stderr[-2000:]


def test_layers_on_two_streams(lib):
    """Calls on two streams take scratch from the same pool at the same time."""
    import torch
    rng = np.random.default_rng(82)
    calls = [moe_call(lib, rng, T, dtype=dt) for T, dt in ((700, "bfloat16"), (1500, "float16"), (9, "float32"))]
    want = [c[0]().clone() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(30):
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                c[0]()
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c[1], w)
    lib.device_status()


def test_scratch_is_given_back_on_request(lib):
    import torch
    call, out, _, _ = moe_call(lib, np.random.default_rng(83), 20000, D=1024)
    torch.cuda.synchronize()
    lib.release_scratch()
    before = torch.cuda.mem_get_info()[0]
    call()
    torch.cuda.synchronize()
    held = before - torch.cuda.mem_get_info()[0]
    assert held >= 20000 * 2 * 1024 * 4                                  # the slots' outputs, kept for the next call
    lib.release_scratch()
    assert before - torch.cuda.mem_get_info()[0] <= held // 8
    want = out.clone()
    assert torch.equal(call(), want)                                     # and taken again
