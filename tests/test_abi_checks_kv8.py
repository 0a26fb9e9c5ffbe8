"""Host-side refusals of the calls of the 8-bit cache, through the C ABI and the binding.

Each case is refused before the library makes any CUDA call; the made-up addresses are never
dereferenced.  The cases run only on machines without a GPU.
"""
import ctypes

import pytest

TQ2_OK, TQ2_EINVAL, TQ2_ESHAPE = 0, 1, 2
A = 0x10000


@pytest.fixture(scope="module")
def bpw():
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses are only passed where no GPU exists")
    import binary_packed_weight_gb300 as bpw
    from binary_packed_weight_gb300 import build
    build.build()
    bpw.load()
    return bpw


def structs(bpw, **change):
    c = dict(codes=A, scales=A, blocks=10, heads=2, tokens=64, dim=128)
    b = dict(table=A, ld=4, offsets=A, lens=A, width=4, seqs=3)
    for k, v in change.items():
        (c if k in c else b)[k] = v
    return ctypes.byref(bpw._Kv8Cache(**c)), ctypes.byref(bpw._Kv8Batch(**b))


CALLS = ["write", "read", "attention"]


def call(bpw, which, c, b, x=A, y=A, dtype=0, T=5, Hq=4, scale=0.1, causal=1, window=0, max_q=0, lse=None):
    lib = bpw.load()
    if which == "attention":
        return lib.kv8_attention(c, b, x, 512, 128, y, 512, 128, dtype, lse, T, Hq, scale, causal, window, max_q, None)
    return getattr(lib, "kv8_" + which)(c, b, x, 256, 128, y, 256, 128, dtype, T, None)


@pytest.mark.parametrize("which", CALLS)
def test_pointers(bpw, which):
    c, b = structs(bpw)
    assert call(bpw, which, None, b) == TQ2_EINVAL and call(bpw, which, c, None) == TQ2_EINVAL
    assert call(bpw, which, c, b, x=None) == TQ2_EINVAL and call(bpw, which, c, b, y=None) == TQ2_EINVAL
    for k in ("codes", "scales", "table", "offsets", "lens"):
        assert call(bpw, which, *structs(bpw, **{k: None})) == TQ2_EINVAL, k
    for k, off in (("codes", 8), ("scales", 2), ("table", 1), ("offsets", 2), ("lens", 2)):
        assert call(bpw, which, *structs(bpw, **{k: A + off})) == TQ2_EINVAL, k
        assert "aligned" in bpw.load().tq2_last_error().decode()
    for dtype, off in ((0, 2), (1, 1), (2, 1)):
        assert call(bpw, which, c, b, x=A + off, dtype=dtype) == TQ2_EINVAL
        assert call(bpw, which, c, b, y=A + off, dtype=dtype) == TQ2_EINVAL
    for dtype in (-1, 3):
        assert call(bpw, which, c, b, dtype=dtype) == TQ2_EINVAL
    assert call(bpw, which, c, b, T=0, x=None, y=None) == TQ2_OK      # nothing to do


@pytest.mark.parametrize("which", CALLS)
def test_shapes(bpw, which):
    for change in (dict(tokens=8), dict(tokens=48), dict(tokens=256), dict(tokens=0), dict(tokens=-16), dict(dim=32), dict(dim=96),
                   dict(dim=256), dict(heads=0), dict(heads=1025), dict(blocks=0), dict(blocks=1 << 23), dict(blocks=1 << 40),
                   dict(seqs=0), dict(seqs=-1), dict(width=0), dict(width=5), dict(width=1 << 25, ld=1 << 25)):
        assert call(bpw, which, *structs(bpw, **change)) == TQ2_ESHAPE, change
    c, b = structs(bpw)
    assert call(bpw, which, c, b, T=-1) == TQ2_ESHAPE
    assert call(bpw, which, c, b, T=1 << 31) == TQ2_ESHAPE


def test_attention_options(bpw):
    c, b = structs(bpw)
    for Hq in (0, 1, 3, -2):
        assert call(bpw, "attention", c, b, Hq=Hq) == TQ2_ESHAPE, Hq
    assert call(bpw, "attention", c, b, T=1 << 29, Hq=4) == TQ2_ESHAPE
    one = structs(bpw, heads=1)                              # rows whose positions less a window pass 32 bits
    assert call(bpw, "attention", *one, T=(1 << 30) + 1, Hq=1, window=(1 << 30) - 1) == TQ2_ESHAPE
    assert "2^30" in bpw.load().tq2_last_error().decode()
    for options in (dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2), dict(causal=-1), dict(window=-1),
                    dict(window=3, causal=0), dict(max_q=-1)):
        assert call(bpw, "attention", c, b, **options) == TQ2_EINVAL, options
    assert call(bpw, "attention", c, b, lse=A + 2) == TQ2_EINVAL


def test_binding_refuses_what_does_not_fit(bpw):
    import torch
    codes, scales = torch.zeros((4, 2, 3, 16, 64), dtype=torch.uint8), torch.zeros((4, 2, 3))
    with pytest.raises(ValueError, match="on the GPU"):
        bpw.KV8Cache(codes, scales)
    with pytest.raises(ValueError, match="blocks, 2, heads"):
        bpw.KV8Cache(codes[:, 0], scales)
    with pytest.raises(ValueError, match="blocks, 2, heads"):
        bpw.KV8Cache(codes[:, :1], scales)
    with pytest.raises(ValueError, match="codes must be contiguous uint8"):
        bpw.KV8Cache(codes.to(torch.int8), scales)
    table, offsets, lens = (torch.zeros(s, dtype=torch.int32) for s in ((2, 5), 3, 2))
    with pytest.raises(ValueError, match="table must be"):
        bpw.KV8Batch(table[0], offsets, lens)
    with pytest.raises(ValueError, match="on the GPU"):
        bpw.KV8Batch(table, offsets, lens)


def test_sizes_whose_products_pass_64_bits_are_refused(bpw):
    """Tables of 2^30 tokens for 2^31 - 1 sequences, and rows near 2^31."""
    c, b = structs(bpw, heads=1024, blocks=1, tokens=16, width=1 << 26, ld=1 << 26, seqs=(1 << 31) - 1)
    assert call(bpw, "attention", c, b, T=(1 << 20) - 1, Hq=2048) == TQ2_ESHAPE
    assert "too many" in bpw.load().tq2_last_error().decode()
