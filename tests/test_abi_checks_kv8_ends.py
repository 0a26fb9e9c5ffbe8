"""Host-side refusals of the 8-bit cache at the ends of the ranges, through the C ABI and the binding.

As in test_abi_checks_kv8.py, the made-up addresses are never dereferenced and the cases run only on
machines without a GPU.
"""
import pytest

from test_abi_checks_kv8 import TQ2_EINVAL, TQ2_ESHAPE, bpw, call, structs  # noqa: F401 (bpw is a fixture)


def test_rows_whose_last_tile_ends_past_32_bits(bpw):  # noqa: F811
    one = structs(bpw, heads=1)
    for T, Hq in (((1 << 30) - 128, 2), ((1 << 30) - 255, 2), ((1 << 31) // 64 - 4, 64)):
        assert (1 << 31) - 512 < T * Hq < 1 << 31
        assert call(bpw, "attention", *one, T=T, Hq=Hq) == TQ2_ESHAPE
        assert "2^31" in bpw.load().tq2_last_error().decode()


def test_more_sequences_than_one_call_walks(bpw):  # noqa: F811
    for seqs in ((1 << 24) + 1, (1 << 31) - 1):
        assert call(bpw, "attention", *structs(bpw, seqs=seqs)) == TQ2_ESHAPE
        assert "sequences are too many" in bpw.load().tq2_last_error().decode()


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_scales_that_no_power_of_two_has(bpw, scale):  # noqa: F811
    assert call(bpw, "attention", *structs(bpw), scale=scale) == TQ2_EINVAL
    assert "finite scale" in bpw.load().tq2_last_error().decode()


class OnGpu:
    """What the binding asks of a tensor, of a tensor that is on no GPU."""

    def __init__(self, t):
        self.t, self.shape, self.dtype, self.is_cuda = t, t.shape, t.dtype, True

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_rows_of_one_element_that_are_one_and_the_same(bpw):  # noqa: F811
    """A table of one block a sequence, the same for all: its rows' stride of 0 is refused like any that is below the width."""
    import torch
    table, offsets, lens = torch.zeros((1, 1), dtype=torch.int32), torch.zeros(6, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    b = bpw.KV8Batch(*(OnGpu(t) for t in (table.expand(5, 1), offsets, lens)))
    assert b._c.ld == 0
    c, _ = structs(bpw)
    assert call(bpw, "attention", c, b._at) == TQ2_ESHAPE
    wide = torch.zeros((5, 7), dtype=torch.int32)
    assert bpw.KV8Batch(*(OnGpu(t) for t in (wide[:, 2:3], offsets, lens)))._c.ld == 7
    assert bpw.KV8Batch(*(OnGpu(t) for t in (wide[:1, 2:3], offsets[:2], lens[:1])))._c.ld == 7
    assert bpw.KV8Batch(*(OnGpu(t) for t in (table.expand(1, 1), offsets[:2], lens[:1])))._c.ld == 1
