"""GPU parity of the 4-bit weights and their products against the f64 oracle.

Packing, dequantization and quantization are bit-exact.  Bound of a product
(derived before its first run): the weights and f16 / bf16 activations are
exact, f32 activations are within 2^-22 |x| + 2^-38 max|x|; a group's sum is
at most 8 steps of 16 products and the groups and k parts at most K/G + 16
additions, each step off by at most 2^-22 of the absolute sum (tensor-core
additions may truncate), then one rounding to the output type.
"""
import numpy as np
import pytest

from oracle import q4 as oq4

pytestmark = pytest.mark.gpu

HALF_ULP = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


def planes(rng, E, N, K, group, zeros):
    codes = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    d = (rng.uniform(0.01, 0.1, (E, N, K // group)) * rng.choice([-1, 1], (E, N, K // group))).astype(np.float16)
    z = rng.integers(0, 16, (E, N, K // group), dtype=np.uint8) if zeros else None
    return codes, d, z


def upload(lib, codes, d, z, group, device="cpu"):
    import torch
    t = [None if a is None else torch.from_numpy(a).to(device) for a in (codes, d, z)]
    return lib.q4_upload(t[0], t[1], t[2], group=group)


def run(lib, w, x, dtype, ldx=0, ldo=0, shift=0):
    """x float64 numpy, rounded to dtype -> (x as the call saw it, out), both float64; ldx, ldo: extra row
    elements; shift: elements the rows start off an aligned address."""
    import torch
    dt = getattr(torch, dtype)
    M = x.shape[0]
    xb = torch.full((M, w.K + ldx + shift), float("nan"), dtype=dt, device="cuda")
    ob = torch.full((M, w.N + ldo + shift), 7.0, dtype=dt, device="cuda")
    xd, out = xb[:, shift:shift + w.K], ob[:, shift:shift + w.N]
    xd.copy_(torch.from_numpy(x).to(dt))
    lib.q4_gemm(w, xd, out)
    lib.device_status()
    o = ob.cpu().double().numpy()
    assert np.all(o[:, :shift] == 7.0) and np.all(o[:, shift + w.N:] == 7.0)       # nothing beside the rows
    return xd.cpu().double().numpy(), o[:, shift:shift + w.N]


def check(got, x, W, K, group, dtype, where):
    ref, scale = oq4.gemm(x, W), oq4.gemm_abs(x, W)
    eps = (8 + K / group + 16) * 2.0 ** -22
    if dtype == "float32":
        eps += 2.0 ** -22
        tail = 2.0 ** -38 * np.abs(x).max(1, keepdims=True) * np.abs(W).sum(1)[None, :]
    else:
        tail = 0.0
    bound = eps * scale + tail + HALF_ULP[dtype] * np.abs(ref) + 2.0 ** -24 * (dtype == "float16")
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{where}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / (scale + 1e-30)):.3g}"


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_dequant_is_exact(lib, group, zeros):
    import torch
    rng = np.random.default_rng(1)
    for E, N, K in ((1, 1, 128), (2, 40, 384), (3, 130, 640)):
        c, d, z = planes(rng, E, N, K, group, zeros)
        for device in ("cpu", "cuda"):
            w = upload(lib, c, d, z, group, device)
            out = torch.full((E, N, K), float("nan"), device="cuda")
            lib.q4_dequant(w, out)
            assert np.array_equal(out.cpu().double().numpy(), oq4.dequant(c, d.view(np.uint16), z, group))


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_quantize_is_exact(lib, group, zeros, dtype):
    import torch
    rng = np.random.default_rng(2)
    w = rng.normal(size=(2, 9, 256)).astype(np.float32)
    w[0, 0] = 0.0                                                     # groups of zeros
    w[0, 1] = np.abs(w[0, 1])                                         # one-sided groups
    w[0, 2] *= 1e-9                                                   # scale below f16's smallest
    wd = torch.from_numpy(w).to(getattr(torch, dtype)).cuda()
    codes = torch.empty((2, 9, 128), dtype=torch.uint8, device="cuda")
    d = torch.empty((2, 9, 256 // group), dtype=torch.float16, device="cuda")
    z = torch.empty((2, 9, 256 // group), dtype=torch.uint8, device="cuda") if zeros else None
    lib.q4_quantize(wd, codes, d, z, group=group)
    rc, rd, rz = oq4.quantize(wd.float().cpu().numpy(), group, zeros)
    assert np.array_equal(d.cpu().numpy().view(np.uint16), rd)
    assert not zeros or np.array_equal(z.cpu().numpy(), rz)
    assert np.array_equal(codes.cpu().numpy(), rc)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False)])
def test_gemm_small_and_ragged(lib, dtype, group, zeros):
    rng = np.random.default_rng(3)
    for N, K in ((1, 128), (7, 384), (16, 256), (40, 1152), (129, 128), (300, 2176)):
        c, d, z = planes(rng, 1, N, K, group, zeros)
        W = oq4.dequant(c, d.view(np.uint16), z, group)[0]
        w = upload(lib, c, d, z, group)
        for M in (1, 2, 3, 5, 8, 9, 16, 17, 33):
            x, got = run(lib, w, rng.normal(size=(M, K)), dtype)
            check(got, x, W, K, group, dtype, f"{M}x{N}x{K}")


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_gemm_k_of_one_group(lib, dtype):
    rng = np.random.default_rng(4)
    for K in (32, 96, 224):
        c, d, z = planes(rng, 1, 50, K, 32, True)
        W = oq4.dequant(c, d.view(np.uint16), z, 32)[0]
        x, got = run(lib, upload(lib, c, d, z, 32), rng.normal(size=(4, K)), dtype)
        check(got, x, W, K, 32, dtype, f"K={K}")


@pytest.mark.parametrize("dtype,M,N,K", [("float32", 1, 4096, 4096), ("bfloat16", 16, 1000, 11008),
                                         ("float16", 11, 700, 14336), ("float32", 7, 513, 8192),
                                         ("float32", 2, 64, 32768), ("bfloat16", 70, 4100, 1024),
                                         ("bfloat16", 4, 20000, 512)])
def test_gemm_wide(lib, dtype, M, N, K):
    """Long rows (fewer activation rows a pass) and many tiles (several units a CTA)."""
    rng = np.random.default_rng(5)
    c, d, z = planes(rng, 1, N, K, 128, True)
    W = oq4.dequant(c, d.view(np.uint16), z, 128)[0]
    x, got = run(lib, upload(lib, c, d, z, 128), rng.normal(size=(M, K)), dtype)
    check(got, x, W, K, 128, dtype, f"{M}x{N}x{K}")


@pytest.mark.parametrize("dtype,M,N,K,group", [("float32", 13, 106, 10624, 128), ("bfloat16", 13, 82, 11136, 64),
                                               ("float32", 16, 33, 4096, 32), ("float16", 16, 300, 32768, 128),
                                               ("float32", 16, 3000, 6176, 32), ("bfloat16", 40, 40, 9600, 128),
                                               ("float32", 9, 16, 32768, 64)])
def test_gemm_rows_longer_than_shared_memory(lib, dtype, M, N, K, group):
    """Several CTAs share a tile's k; their ranges and the last chunk are uneven."""
    rng = np.random.default_rng(13)
    c, d, z = planes(rng, 1, N, K, group, True)
    W = oq4.dequant(c, d.view(np.uint16), z, group)[0]
    w = upload(lib, c, d, z, group)
    for ldx in (0, 3):
        x, got = run(lib, w, rng.normal(size=(M, K)), dtype, ldx)
        check(got, x, W, K, group, dtype, f"{M}x{N}x{K}")


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_gemm_strided_and_unaligned_rows(lib, dtype):
    rng = np.random.default_rng(6)
    c, d, z = planes(rng, 1, 45, 384, 64, True)
    W = oq4.dequant(c, d.view(np.uint16), z, 64)[0]
    w = upload(lib, c, d, z, 64)
    for ldx, ldo, shift in ((8, 8, 0), (3, 5, 0), (0, 0, 1), (7, 2, 3)):
        x, got = run(lib, w, rng.normal(size=(6, 384)), dtype, ldx, ldo, shift)
        check(got, x, W, 384, 64, dtype, f"{ldx},{ldo},{shift}")


@pytest.mark.parametrize("magnitude", [1e-30, 1e-6, 1e4, 1e30])
def test_gemm_f32_scales_of_rows(lib, magnitude):
    """Rows far outside the f16 range, with small entries beside large ones."""
    rng = np.random.default_rng(7)
    c, d, z = planes(rng, 1, 33, 512, 128, False)
    W = oq4.dequant(c, d.view(np.uint16), z, 128)[0]
    x = rng.normal(size=(3, 512)) * magnitude
    x[1] *= 10.0 ** rng.uniform(-6, 0, 512)
    x, got = run(lib, upload(lib, c, d, z, 128), x, "float32")
    check(got, x, W, 512, 128, "float32", f"{magnitude}")


def test_gemm_bf16_range(lib):
    rng = np.random.default_rng(8)
    c, d, z = planes(rng, 1, 33, 512, 128, False)
    W = oq4.dequant(c, d.view(np.uint16), z, 128)[0]
    for magnitude in (1e-20, 1e20):
        x, got = run(lib, upload(lib, c, d, z, 128), rng.normal(size=(3, 512)) * magnitude, "bfloat16")
        check(got, x, W, 512, 128, "bfloat16", f"{magnitude}")


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_gemm_zero_rows_and_nonfinite_rows(lib, dtype):
    rng = np.random.default_rng(9)
    c, d, z = planes(rng, 1, 20, 256, 128, False)
    c[0, 3] = 0x88                                                    # a row of weights that is exactly zero
    W = oq4.dequant(c, d.view(np.uint16), z, 128)[0]
    x = rng.normal(size=(5, 256))
    x[1] = 0.0
    x[2, 17] = np.nan
    x[3, 40] = np.inf
    xs, got = run(lib, upload(lib, c, d, z, 128), x, dtype)
    assert not got[1].any() and np.all(got[[0, 1, 4]][:, 3] == 0.0)
    assert np.all(np.isnan(got[2]))
    assert not np.isfinite(got[3][W[:, 40] != 0]).any()
    good = [0, 1, 4]                                                  # the other rows are not touched by them
    check(got[good], xs[good], W, 256, 128, dtype, "rows beside non-finite ones")


def test_gemm_no_rows_and_refusals(lib):
    import torch
    rng = np.random.default_rng(10)
    c, d, z = planes(rng, 1, 20, 256, 128, False)
    w = upload(lib, c, d, z, 128)
    x, out = torch.zeros((0, 256), device="cuda"), torch.zeros((0, 20), device="cuda")
    lib.q4_gemm(w, x, out)
    x, out = torch.zeros((2, 256), device="cuda"), torch.zeros((2, 20), device="cuda")
    with pytest.raises(ValueError):
        lib.q4_gemm(w, x[:, :128], out)
    with pytest.raises(ValueError):
        lib.q4_gemm(w, x.t().contiguous().t(), out)
    with pytest.raises(TypeError):
        lib.q4_gemm(w, x.half(), out)
    with pytest.raises(TypeError):
        lib.q4_gemm(w, x.double(), out.double())
    two = upload(lib, *planes(rng, 2, 20, 256, 128, False), 128)
    with pytest.raises(lib.TQ2Error) as info:
        lib.q4_gemm(two, x, out)
    assert info.value.status == 2
    with pytest.raises(ValueError):
        lib.q4_upload(torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 3), dtype=torch.float16), group=32)
    with pytest.raises(lib.TQ2Error):
        lib.q4_upload(torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((4, 16), dtype=torch.float16), group=16)


def test_gemm_repeats_bit_for_bit_and_on_another_stream(lib):
    import torch
    rng = np.random.default_rng(11)
    c, d, z = planes(rng, 1, 700, 2048, 128, True)
    w = upload(lib, c, d, z, 128)
    x = torch.randn((9, 2048), device="cuda")
    outs = []
    for i in range(4):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            y = x * 1.0                                               # written on the stream the call is on
            o = torch.empty((9, 700), device="cuda")
            lib.q4_gemm(w, y, o)
        torch.cuda.current_stream().wait_stream(s)
        outs.append(o.cpu())
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_gemm_in_a_graph(lib):
    import torch
    rng = np.random.default_rng(12)
    c, d, z = planes(rng, 1, 128, 512, 64, False)
    w = upload(lib, c, d, z, 64)
    x, out = torch.randn((3, 512), device="cuda"), torch.empty((3, 128), device="cuda")
    lib.q4_gemm(w, x, out)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.q4_gemm(w, x, out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_gemm_beyond_32_bit_offsets(lib):
    """17 GB of codes in rows too long for shared memory, more columns than a cluster's sums fit in."""
    import torch
    N, K, group = (1 << 20) - 5, 32768, 128
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    gen = torch.Generator(device="cuda").manual_seed(13)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    d = torch.rand((N, K // group), device="cuda", generator=gen).mul_(0.1).half()
    w = lib.q4_upload(codes, d, None, group=group)
    rows = np.unique(np.concatenate([[0, 1, N - 1], np.random.default_rng(14).integers(0, N, 60)]))
    pick = torch.from_numpy(rows).cuda()
    W = oq4.dequant(codes[pick].cpu().numpy()[None], d[pick].cpu().numpy().view(np.uint16)[None], None, group)[0]
    del codes, d
    for dtype, M in (("float32", 2), ("bfloat16", 3)):
        x = torch.randn((M, K), device="cuda", generator=gen).to(getattr(torch, dtype))
        out = lib.q4_gemm(w, x, torch.empty((M, N), dtype=x.dtype, device="cuda"))
        lib.device_status()
        check(out[:, pick].cpu().double().numpy(), x.cpu().double().numpy(), W, K, group, dtype, "sampled rows")
        assert bool(torch.isfinite(out).all())
    w.free()
