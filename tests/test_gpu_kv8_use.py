"""The 8-bit cache as a serving program uses it: prompts and then tokens, in graphs, on several streams."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest

from kv8_util import Cache, attention_of, check_attention, queries
from oracle import kv8

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("prompt,decoded", [(1, 1), (100, 5), (300, 40)])
def test_decode_layer_example(lib, prompt, decoded):
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    errors = m.main(prompt, decoded)
    # bf16 outputs: half an ulp is at most 2^-8 of each value; the attention's weights are rounded to f16 too
    assert errors["projection"] < 2.0 ** -8 and errors["attention"] < 2.0 ** -8 + 2.0 ** -11


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_prompts_then_tokens(lib, dtype):
    """Written codes follow the oracle over prompts, chunks and single tokens; each step's attention is right."""
    import torch
    rng = np.random.default_rng(60)
    dt = getattr(torch, dtype)
    H, G, D, B = 2, 3, 64, 16
    final = [90, 41, 70]
    c = Cache(lib, rng, final, [0, 0, 0], H=H, D=D, B=B)
    start = [33, 1, 50]
    steps = [start] + [[33 + 20, 1, 50 + 7]] + [[53 + i, 1 + i, 57] for i in range(1, 18)]
    done = [0, 0, 0]
    for lens in steps:
        n = [b - a for a, b in zip(done, lens)]
        done = lens
        c.lens[:], c.offsets[:], c.T = lens, np.concatenate(([0], np.cumsum(n))), sum(n)
        c.upload()
        c.batch = lib.KV8Batch(c.d["table"], c.d["offsets"], c.d["lens"])
        k, v = (torch.from_numpy(rng.normal(size=(c.T, H, D)) * 2.0 ** rng.uniform(-2, 2, (c.T, 1, 1))).to(dt).cuda() for _ in range(2))
        want = kv8.write(c.codes, c.scales, c.table, c.offsets, c.lens, np.stack((k.float().cpu().numpy(), v.float().cpu().numpy())))
        lib.kv8_write(c.cache, c.batch, k, v)
        lib.device_status()
        c.codes, c.scales = c.on_gpu()
        assert np.array_equal(c.codes, want[0]) and np.array_equal(c.scales, want[1])
        q, out, lse = c.attend(queries(rng, c.T, H * G, D), dtype)
        check_attention(out, lse, attention_of(c, q), dtype, D, max(lens), str(lens))


def step_call(lib, rng, n, dtype="bfloat16", S=5, L=500, H=2, G=4, D=128, B=64):
    """A step of S sequences (write and attention) whose lengths live on the GPU: (call, out, lse, lens)."""
    import torch
    dt = getattr(torch, dtype)
    c = Cache(lib, rng, [L] * S, [n] * S, H=H, D=D, B=B)
    T = S * n
    k, v = (torch.from_numpy(rng.normal(size=(T, H, D))).to(dt).cuda() for _ in range(2))
    q = torch.from_numpy(rng.normal(size=(T, H * G, D))).to(dt).cuda()
    out, lse = torch.empty_like(q), torch.empty((T, H * G), device="cuda")
    c.d["lens"].fill_(n + 37)

    def call():
        lib.kv8_write(c.cache, c.batch, k, v)
        lib.kv8_attention(c.cache, c.batch, q, out, lse)
    return call, out, lse, c


@pytest.mark.parametrize("n,dtype", [(1, "bfloat16"), (1, "float32"), (3, "float16"), (150, "bfloat16"), (150, "float32")])
def test_step_in_a_graph_follows_the_lengths(lib, n, dtype):
    """Captured once; the lengths move on the GPU between replays."""
    import torch
    call, out, lse, c = step_call(lib, np.random.default_rng(61), n, dtype)
    codes, scales, lens = c.d["codes"].clone(), c.d["scales"].clone(), c.d["lens"].clone()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    want = []
    for start in (lens, lens + 60, lens + 200):
        c.d["codes"].copy_(codes), c.d["scales"].copy_(scales), c.d["lens"].copy_(start)
        call()
        want.append((out.clone(), lse.clone(), c.d["codes"].clone(), c.d["scales"].clone()))
    for start, w in zip((lens, lens + 60, lens + 200), want):
        c.d["codes"].copy_(codes), c.d["scales"].copy_(scales), c.d["lens"].copy_(start)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for got, x in zip((out, lse, c.d["codes"], c.d["scales"]), w):
            assert torch.equal(got, x)
    lib.device_status()


FIRST = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import numpy as np, torch
import binary_packed_weight_gb300 as lib
from test_gpu_kv8_use import step_call
call, out, lse, c = step_call(lib, np.random.default_rng(62), {n})
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
got = out.clone(), lse.clone()
call()
assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
lib.device_status()
print("as captured")
"""


@pytest.mark.parametrize("n", [1, 200])
def test_first_call_of_a_process_may_be_captured(lib, n):
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, n=n)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as captured" in r.stdout, r.stderr[-2000:]


def test_steps_and_graphs_on_several_streams(lib):
    """Calls of both paths take scratch from one pool at the same time, eager and replayed."""
    import torch
    rng = np.random.default_rng(63)
    made = [step_call(lib, rng, n, dt) for n, dt in ((1, "bfloat16"), (200, "float16"), (2, "float32"), (300, "bfloat16"))]
    want = []
    for call, out, lse, _ in made:
        call()
        want.append((out.clone(), lse.clone()))
    torch.cuda.synchronize()
    graphs = []
    for call, *_ in made[2:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    runs = [made[0][0], made[1][0], graphs[0].replay, graphs[1].replay]
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(25):
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                r()
    torch.cuda.synchronize()
    for (_, out, lse, _), (o, l) in zip(made, want):
        assert torch.equal(out, o) and torch.equal(lse, l)
    lib.device_status()


def test_a_bound_of_rows_that_is_too_low_is_only_slower(lib):
    rng = np.random.default_rng(64)
    c = Cache(lib, rng, [300, 20], [170, 3], H=2, D=64, B=32)
    q, out, lse = c.attend(queries(rng, c.T, 8, 64), "bfloat16", max_q=1)
    check_attention(out, lse, attention_of(c, q), "bfloat16", 64, 300)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_decoded_sequences_beside_long_ones_in_large_tables(lib, dtype):
    """Tables that hold much: few rows go the streaming way, many the tensor cores', in one call."""
    rng = np.random.default_rng(65)
    lens, n = [600, 40, 300, 900, 0, 77], [1, 40, 200, 2, 0, 8]
    c = Cache(lib, rng, lens, n, H=2, D=64, B=16, width=6000)
    assert len(lens) * 6000 * 16 * 2 * 64 * 2 > 32 << 20
    for options in ({}, {"window": 100}):
        q, out, lse = c.attend(queries(rng, c.T, 8, 64), dtype, pad=2, **options)
        check_attention(out, lse, attention_of(c, q, **options), dtype, 64, 900)


@pytest.mark.parametrize("rows", [8, 9, 16, 17, 32, 33, 128, 129, 256, 257])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_rows_on_both_sides_of_each_choice(lib, dtype, rows):
    """One query with as many heads as rows: tiles of 8, 16, 128 and 256, and the change of path."""
    rng = np.random.default_rng(66)
    c = Cache(lib, rng, [333, 64], [1, 1], H=1, D=128, B=64)
    q, out, lse = c.attend(queries(rng, 2, rows, 128), dtype)
    check_attention(out, lse, attention_of(c, q), dtype, 128, 333)
