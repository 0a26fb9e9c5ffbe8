"""Host-side argument checks of the 4-bit and mixture-of-experts calls, through the C ABI.

Each case is refused before the library makes any CUDA call.  The non-null
pointers are made-up addresses that are never dereferenced; as in
test_abi_checks.py the cases run only on machines without a GPU.
"""
import ctypes

import pytest

TQ2_OK, TQ2_EINVAL, TQ2_ESHAPE = 0, 1, 2
A = 0x10000


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses are only passed where no GPU exists")
    import binary_packed_weight_gb300 as bpw
    from binary_packed_weight_gb300 import build
    build.build()
    return bpw.load()


def _err(lib):
    return lib.tq2_last_error().decode()


def test_q4_upload(lib):
    h = ctypes.c_void_p(123)
    out = ctypes.byref(h)
    for args in ((None, A, None), (A, None, None)):
        assert lib.q4_upload(*args, 1, 16, 128, 128, out, None) == TQ2_EINVAL
        assert h.value is None
    assert lib.q4_upload(A, A, None, 1, 16, 128, 128, None, None) == TQ2_EINVAL
    for E, N, K, g in ((0, 16, 128, 128), (1025, 16, 128, 128), (1, 0, 128, 128), (1, 16, 0, 128), (1, 16, 96, 128),
                       (1, 16, 128, 16), (1, 16, 128, 256), (1, 16, 32896, 128), (1, (1 << 24) + 1, 128, 128),
                       (1, 1 << 24, 32768, 128)):
        assert lib.q4_upload(A, A, None, E, N, K, g, out, None) == TQ2_ESHAPE, (E, N, K, g)
    assert lib.q4_upload(A + 1, A, None, 1, 16, 128, 128, out, None) == TQ2_EINVAL
    assert "aligned" in _err(lib)
    assert lib.q4_free(None) == TQ2_OK
    assert lib.q4_shape(None, None, None, None, None) == TQ2_EINVAL
    assert lib.q4_dequant(None, A, None) == TQ2_EINVAL


def test_q4_quantize(lib):
    assert lib.q4_quantize(None, 0, 1, 128, 128, A, A, None, None) == TQ2_EINVAL
    assert lib.q4_quantize(A, 0, 1, 128, 128, None, A, None, None) == TQ2_EINVAL
    assert lib.q4_quantize(A, 3, 1, 128, 128, A, A, None, None) == TQ2_EINVAL
    assert lib.q4_quantize(A, 0, 1, 128, 128, A + 2, A, None, None) == TQ2_EINVAL
    assert lib.q4_quantize(A + 2, 0, 1, 128, 128, A, A, None, None) == TQ2_EINVAL
    for rows, K, g in ((0, 128, 128), (1, 100, 32), (1, 128, 48), (1, 0, 32), (1 << 35, 128, 128)):
        assert lib.q4_quantize(A, 0, rows, K, g, A, A, None, None) == TQ2_ESHAPE, (rows, K, g)


def test_q4_gemm(lib):
    assert lib.q4_gemm(None, A, 128, A, 16, 0, 1, None) == TQ2_EINVAL
    # refused (or done) before the handle is read
    assert lib.q4_gemm(A, A, 128, A, 16, 7, 1, None) == TQ2_EINVAL
    assert lib.q4_gemm(A, A, 128, A, 16, 0, -1, None) == TQ2_ESHAPE
    assert lib.q4_gemm(A, A, 128, A, 16, 0, (1 << 20) + 1, None) == TQ2_ESHAPE
    assert lib.q4_gemm(A, A, 128, A, 16, 0, 0, None) == TQ2_OK
    assert lib.q4_gemm(A, None, 128, A, 16, 0, 1, None) == TQ2_EINVAL


def _route(lib, T=4, E=8, k=2, ld=8, dtype=0, score=0, groups=1, top=1, scale=1.0, logits=A, off=A, slots=A):
    return lib.moe_route(logits, ld, dtype, None, T, E, k, score, groups, top, 1, scale, A, A, off, slots, None)


def test_moe_route(lib):
    assert _route(lib, logits=None) == TQ2_EINVAL
    assert _route(lib, dtype=3) == TQ2_EINVAL
    assert _route(lib, score=2) == TQ2_EINVAL
    assert _route(lib, scale=float("inf")) == TQ2_EINVAL
    assert _route(lib, scale=float("nan")) == TQ2_EINVAL
    assert _route(lib, off=None) == TQ2_EINVAL
    assert _route(lib, slots=None) == TQ2_EINVAL
    for bad in (dict(T=-1), dict(E=0, ld=1), dict(E=1025, ld=1025), dict(k=0), dict(k=9), dict(ld=7),
                dict(groups=3), dict(groups=0), dict(groups=4, top=5), dict(groups=4, top=0),
                dict(E=64, ld=64, groups=64), dict(T=(1 << 23) + 1), dict(E=64, ld=64, k=33)):
        assert _route(lib, **bad) == TQ2_ESHAPE, bad
    for bad in (dict(logits=A + 2), dict(logits=A + 1, dtype=2), dict(off=A + 2), dict(slots=A + 1)):
        assert _route(lib, **bad) == TQ2_EINVAL and "aligned" in _err(lib), bad
    assert _route(lib, T=0, off=None, slots=None) == TQ2_OK


def test_moe_route_backward(lib):
    def back(T=4, E=8, k=2, ld=8, ldd=8, dtype=0, score=0, scale=1.0, logits=A, dl=A):
        return lib.moe_route_backward(logits, ld, dtype, None, A, A, dl, ldd, T, E, k, score, 1, scale, None)
    assert back(logits=None) == TQ2_EINVAL
    assert back(dl=None) == TQ2_EINVAL
    assert back(dtype=-1) == TQ2_EINVAL
    assert back(score=5) == TQ2_EINVAL
    for bad in (dict(ld=7), dict(ldd=7), dict(k=9), dict(T=-1), dict(E=2000, ld=2000, ldd=2000)):
        assert back(**bad) == TQ2_ESHAPE, bad
    assert back(logits=A + 2) == TQ2_EINVAL and back(dl=A + 1, dtype=1) == TQ2_EINVAL
    assert back(T=0) == TQ2_OK


def test_moe_experts(lib):
    def experts(gate=A, T=4, k=2, dtype=0):
        return lib.moe_experts(gate, A, A, A, 64, dtype, A, A, A, A, A, 64, T, k, None)
    assert experts(gate=None) == TQ2_EINVAL
    assert experts(dtype=9) == TQ2_EINVAL
    for bad in (dict(T=-1), dict(k=0), dict(k=33), dict(T=1 << 24), dict(T=1 << 62, k=4)):      # refused before a handle is read
        assert experts(**bad) == TQ2_ESHAPE, bad


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    import torch
    import binary_packed_weight_gb300 as bpw
    w = bpw.Q4Weight(None, 1, 16, 128, 128)
    x, out = torch.zeros((2, 128)), torch.zeros((2, 16))
    with pytest.raises(ValueError, match="on the GPU"):
        bpw.q4_gemm(w, x, out)
    with pytest.raises(ValueError, match=r"x must be \[2, 128\]"):
        bpw.q4_gemm(w, x[:, :64], out)
    with pytest.raises(TypeError):
        bpw.q4_gemm(w, x.half(), out)
    with pytest.raises(ValueError, match="on the GPU"):
        bpw.q4_dequant(w, torch.zeros((1, 16, 128)))
    with pytest.raises(ValueError, match="on the GPU"):
        bpw.q4_quantize(x, torch.zeros((2, 64), dtype=torch.uint8), torch.zeros((2, 1), dtype=torch.float16))
    ids, wt = torch.zeros((2, 4), dtype=torch.int32), torch.zeros((2, 4))
    with pytest.raises(ValueError, match="on the GPU"):
        bpw.moe_route(out, ids, wt)
    with pytest.raises(ValueError, match="score"):
        bpw._score("tanh", "moe_route")
    with pytest.raises(ValueError, match="on the GPU"):
        bpw.moe_route_backward(out, ids, wt, torch.zeros_like(out))
    with pytest.raises(ValueError, match="on the GPU"):
        bpw.moe_experts(w, w, w, x, ids, wt, torch.zeros(2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                        torch.zeros_like(x))


def test_binding_refuses_groups_that_divide_nothing(lib):
    import torch
    import binary_packed_weight_gb300 as bpw
    codes, scales = torch.zeros((2, 64), dtype=torch.uint8), torch.zeros((2, 1), dtype=torch.float16)
    for group in (0, -32):
        with pytest.raises(ValueError, match="group must be"):
            bpw.q4_upload(codes, scales, group=group)
        with pytest.raises(ValueError, match="group must be"):
            bpw.q4_quantize(torch.zeros((2, 128)), codes, scales, group=group)
    with pytest.raises(ValueError, match="scalar"):
        bpw.q4_quantize(torch.zeros(()), codes, scales)


@pytest.mark.parametrize("kind", ["q4", "tq2"])
def test_a_handle_is_freed_once_whatever_the_library_reports(lib, monkeypatch, kind):
    """The library deletes a handle before it reports that its memory could not be freed."""
    import binary_packed_weight_gb300 as bpw
    freed = []

    class Failing:
        tq2_last_error = staticmethod(lambda: b"planted")
        tq2_status_string = staticmethod(lambda status: b"CUDA error")
        q4_free = staticmethod(lambda h: freed.append(h) or 4)
        tq2_free = q4_free
    monkeypatch.setattr(bpw, "_lib", Failing)
    w = bpw.Q4Weight(A, 1, 16, 128, 128) if kind == "q4" else bpw.Weight(A, 16, 128)
    with pytest.raises(bpw.TQ2Error):
        w.free()
    w.free()
    del w
    assert freed == [A]
