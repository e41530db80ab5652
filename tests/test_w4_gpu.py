"""Products with 4-bit weights against 64-bit products with the matrix that the
codes, scales and zero points stand for.

Tolerance.  Each product x * (q - z) * s is formed from at most three parts of x
(which add up to x exactly), as a sum over q and one over z; every part meets at most
3K additions, and three roundings more (the correction by z, the scale, the sum over
parts).  With |terms| = |x| * s * (q + z) the result is therefore within
1.01 * (3K + 8) * 2^-24 * sum |terms| in any order.  Small integers with scales that
are powers of two are exact in every order and compared bitwise."""
import itertools

import numpy as np
import pytest

import dense_fp32_matrix_f32_amd as sg
from gpu_helpers import log, torch_cuda

pytestmark = pytest.mark.gpu

SENT = float(np.float32(-7.25e30))
TYPES = ("float32", "float16", "bfloat16")


def make(rng, experts, K, N, group, zeros, exact, scale_type):
    """(codes as given to w4_pack, scales and zeros as torch tensors, the matrices and
    |s| * (q + z) in 64 bits)."""
    torch = torch_cuda()
    groups = -(-K // group)
    q = rng.integers(0, 16, (experts, K, N)).astype(np.uint8)
    z = rng.integers(0, 16, (experts, groups, N)).astype(np.uint8) if zeros else None
    if exact:
        s = 2.0 ** rng.integers(-3, 3, (experts, groups, N))
    else:
        s = rng.uniform(0.001, 0.1, (experts, groups, N)) * rng.choice([-1, 1], (experts, groups, N))
    st = torch.from_numpy(s).to(getattr(torch, scale_type))
    s = st.double().numpy()
    full = np.zeros((experts, K + K % 2, N), np.uint8)
    full[:, :K] = q
    if K % 2:
        full[:, K] = rng.integers(0, 16, (experts, N))  # the half byte past K counts for nothing
    codes = full[:, 0::2] | (full[:, 1::2] << 4)
    sk = np.repeat(s, group, 1)[:, :K]
    zk = np.repeat(z, group, 1)[:, :K].astype(np.float64) if zeros else np.full((experts, K, N), 8.0)
    return (torch.from_numpy(codes).cuda(), st.cuda(), torch.from_numpy(z).cuda() if zeros else None,
            sk * (q - zk), np.abs(sk) * (q + zk))


def close(got, want, K, mag, what):
    off = np.abs(got.double().cpu().numpy() - want)
    limit = 1.01 * (3 * K + 8) * 2.0**-24 * mag + 1e-37
    bad = off > limit
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, the worst by "
                           f"{float((off / limit).max()):.3g} of the bound")


def buffer(torch, rows, cols, pad, offset):
    buf = torch.full((rows * (cols + pad) + offset + 8,), SENT, device="cuda")
    return buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def run(x, w, offsets=None, pad=0, offset=0):
    """The product into a padded buffer whose padding is checked; rows on the device."""
    torch = torch_cuda()
    rows = x.shape[0]
    out, buf = buffer(torch, rows, w.N, pad, offset)
    a, _ = buffer(torch, rows, w.K, pad, offset)
    a.copy_(torch.from_numpy(x))
    sg.matmul_w4(a, w, offsets=offsets, out=out)
    got = out.clone()
    out.fill_(SENT)
    assert int((buf != SENT).sum()) == 0, "wrote outside C"
    return got


ROWS = [1, 2, 3, 5, 6, 10, 11, 16, 17, 33, 64, 100]
SHAPES = [(1, 1), (15, 31), (16, 32), (17, 33), (64, 128), (40, 129), (100, 255), (257, 1000),
          (33, 2048), (128, 1100)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128, 256, 1024])
def test_product(N, K, group):
    torch = torch_cuda()
    rng = np.random.default_rng(N * 1000 + K + group)
    for i, rows in enumerate(ROWS):
        for exact in (True, False):
            zeros, scale_type = bool((i + exact) % 2), TYPES[(i + group // 32) % 3]
            log(f"[gpu] w4 {rows} x {N} x {K} group {group} {scale_type} zeros {zeros} exact {exact}")
            codes, s, z, W, mag = make(rng, 1, K, N, group, zeros, exact, scale_type)
            w = sg.w4_pack(codes[0], s[0], None if z is None else z[0], K=K, group=group)
            x = rng.integers(-4, 5, (rows, K)).astype(np.float32) if exact else \
                (rng.standard_normal((rows, K)) * 10.0 ** rng.integers(-3, 4, (rows, 1))).astype(np.float32)
            got = run(x, w, pad=(0, 3, 4)[i % 3], offset=(0, 1, 4)[i % 3])
            want = x.astype(np.float64) @ W[0]
            if exact:
                assert np.array_equal(got.double().cpu().numpy(), want)
            else:
                close(got, want, K, np.abs(x.astype(np.float64)) @ mag[0], "w4")


@pytest.mark.parametrize("rows,N,K", [(1, 4096, 4096), (4, 4097, 1023), (12, 1000, 8192),
                                      (40, 2048, 2048), (300, 520, 700), (1024, 260, 512)])
def test_product_of_ordinary_sizes(rows, N, K):
    torch = torch_cuda()
    rng = np.random.default_rng(rows)
    for group, zeros, scale_type in [(128, False, "float16"), (32, True, "bfloat16")]:
        log(f"[gpu] w4 {rows} x {N} x {K} group {group}")
        codes, s, z, W, mag = make(rng, 1, K, N, group, zeros, False, scale_type)
        w = sg.w4_pack(codes[0], s[0], None if z is None else z[0], K=K, group=group)
        x = rng.standard_normal((rows, K)).astype(np.float32)
        close(run(x, w), x.astype(np.float64) @ W[0], K, np.abs(x.astype(np.float64)) @ mag[0], "w4")


@pytest.mark.parametrize("rows,N,K,group", [
    (1000, 1500, 300, 32), (4100, 1000, 300, 32), (4111, 1023, 140, 32), (6200, 256, 4, 32),
    (1001, 1500, 300, 256), (600, 2047, 129, 64),                          # 16 x 128
    (801, 2047, 129, 64), (2100, 2000, 200, 64), (2081, 1999, 385, 256),
    (513, 2900, 1030, 128),                                                # 16 x 256
    (1001, 2047, 140, 32), (2030, 1000, 300, 32),                          # 32 x 256
    (2048, 2000, 200, 64), (2019, 1999, 385, 256)])                        # 32 x 512
def test_product_of_many_rows(rows, N, K, group):
    """Sizes at which the kernels for many rows run, from one work-group a CU on."""
    torch = torch_cuda()
    rng = np.random.default_rng(rows)
    for zeros, scale_type, exact in [(True, "float32", True), (False, "bfloat16", False),
                                     (True, "float16", False)]:
        log(f"[gpu] w4 {rows} x {N} x {K} group {group} {scale_type} zeros {zeros}")
        codes, s, z, W, mag = make(rng, 1, K, N, group, zeros, exact, scale_type)
        w = sg.w4_pack(codes[0], s[0], None if z is None else z[0], K=K, group=group)
        x = rng.integers(-4, 5, (rows, K)).astype(np.float32) if exact else \
            rng.standard_normal((rows, K)).astype(np.float32)
        got = run(x, w, pad=1, offset=3)
        if exact:
            assert np.array_equal(got.double().cpu().numpy(), x.astype(np.float64) @ W[0])
        else:
            close(got, x.astype(np.float64) @ W[0], K, np.abs(x.astype(np.float64)) @ mag[0], "w4")


@pytest.mark.parametrize("which", ["one has all", "ragged", "rows of no expert"])
@pytest.mark.parametrize("rows,N,experts,group", [(1000, 1300, 16, 64), (500, 1300, 16, 128),
                                                  (2200, 1500, 4, 64), (2200, 700, 4, 32)])
def test_product_of_many_rows_by_expert(rows, N, experts, group, which):
    torch = torch_cuda()
    K = 200
    rng = np.random.default_rng(5)
    offsets = [int(o) for o in OFFSETS[which](rows, experts)]
    codes, s, z, W, mag = make(rng, experts, K, N, group, True, True, "float16")
    w = sg.w4_pack(codes, s, z, K=K, group=group)
    x = rng.integers(-4, 5, (rows, K)).astype(np.float32)
    got = run(x, w, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), pad=3)
    want = np.full((rows, N), SENT)
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        want[lo:hi] = x[lo:hi].astype(np.float64) @ W[e]
    assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 7, 8])
def test_product_of_very_few_k(K):
    torch = torch_cuda()
    rng = np.random.default_rng(K)
    for rows, N in [(1, 5), (3, 40), (7, 300), (20, 17), (70, 33)]:
        for zeros in (False, True):
            codes, s, z, W, _ = make(rng, 2, K, N, 32, zeros, True, "float32")
            w = sg.w4_pack(codes, s, z, K=K, group=32)
            x = rng.integers(-4, 5, (rows, K)).astype(np.float32)
            lo = rows // 3
            got = run(x, w, offsets=torch.tensor([0, lo, rows], dtype=torch.int32, device="cuda"), pad=2)
            want = np.concatenate([x[:lo].astype(np.float64) @ W[0], x[lo:].astype(np.float64) @ W[1]])
            assert np.array_equal(got.double().cpu().numpy(), want)


OFFSETS = {"each one row": lambda R, E: [min(e, R) for e in range(E + 1)],
           "one has all": lambda R, E: [0] * (E // 2 + 1) + [R] * (E - E // 2),
           "ragged": lambda R, E: [0] + sorted(np.random.default_rng(R).integers(0, R + 1, E - 1)) + [R],
           "rows of no expert": lambda R, E: [R // 5 + (R - R // 5 - R // 4) * e // E for e in range(E + 1)]}


@pytest.mark.parametrize("which", list(OFFSETS))
@pytest.mark.parametrize("rows,N,K,experts", [(1, 20, 40, 1), (3, 64, 128, 8), (8, 130, 257, 64),
                                              (40, 48, 300, 5), (100, 33, 512, 3), (65, 16, 128, 130),
                                              (200, 200, 64, 6)])
def test_product_by_expert(rows, N, K, experts, which):
    torch = torch_cuda()
    rng = np.random.default_rng(rows * 7 + N)
    offsets = [int(o) for o in OFFSETS[which](rows, experts)]
    dev = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for (group, zeros, scale_type), exact in itertools.product(
            [(32, True, "float16"), (64, False, "float32"), (128, True, "bfloat16")], (True, False)):
        log(f"[gpu] w4 by expert {rows} x {N} x {K}, {experts} experts, {which}, group {group}")
        codes, s, z, W, mag = make(rng, experts, K, N, group, zeros, exact, scale_type)
        w = sg.w4_pack(codes, s, z, K=K, group=group)
        x = rng.integers(-4, 5, (rows, K)).astype(np.float32) if exact else \
            rng.standard_normal((rows, K)).astype(np.float32)
        got = run(x, w, offsets=dev, pad=3, offset=1)
        want, m = np.full((rows, N), SENT), np.zeros((rows, N))
        for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            want[lo:hi] = x[lo:hi].astype(np.float64) @ W[e]
            m[lo:hi] = np.abs(x[lo:hi].astype(np.float64)) @ mag[e]
        want = want.astype(np.float32).astype(np.float64) if exact else want
        if exact:
            assert np.array_equal(got.double().cpu().numpy(), want)
        else:
            own = np.zeros(rows, bool)
            own[offsets[0]:offsets[-1]] = True
            close(got[torch.from_numpy(own).cuda()], want[own], K, m[own], "w4 by expert")
            assert (got[torch.from_numpy(~own).cuda()] == SENT).all()


def test_offsets_out_of_the_rows_are_clamped():
    torch = torch_cuda()
    rng = np.random.default_rng(1)
    codes, s, z, W, mag = make(rng, 3, 64, 40, 32, False, True, "float32")
    w = sg.w4_pack(codes, s, z, K=64, group=32)
    x = rng.integers(-4, 5, (50, 64)).astype(np.float32)
    for bad, spans in [([0, 1000, 2**31 - 1, -5], [(0, 50), (50, 50), (50, 50)]),
                       ([-2**31, -1, 20, 30], [(0, 0), (0, 20), (20, 30)]),
                       ([40, 20, 10, 400], [(40, 40), (20, 20), (10, 50)])]:
        got = run(x, w, offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        want = np.full((50, 40), np.float32(SENT), np.float64)
        for e, (lo, hi) in enumerate(spans):
            want[lo:hi] = x[lo:hi].astype(np.float64) @ W[e]
        assert np.array_equal(got.double().cpu().numpy(), want)


def test_no_rows_columns_or_k():
    torch = torch_cuda()
    z8 = torch.zeros((0, 20), dtype=torch.uint8, device="cuda")
    w = sg.w4_pack(z8, torch.zeros((0, 20), device="cuda"), K=0, group=32)
    out = torch.full((3, 20), SENT, device="cuda")
    assert sg.matmul_w4(torch.empty((3, 0), device="cuda"), w, out=out).eq(0).all()
    off = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    out.fill_(SENT)
    sg.matmul_w4(torch.empty((3, 0), device="cuda"), w, offsets=off, out=out)
    assert out[1].eq(0).all() and out[0].eq(SENT).all() and out[2].eq(SENT).all()
    w = sg.w4_quantize(torch.ones((64, 20), device="cuda"), group=32)
    assert sg.matmul_w4(torch.empty((0, 64), device="cuda"), w).shape == (0, 20)
    w = sg.w4_quantize(torch.ones((64, 0), device="cuda"), group=32)
    assert sg.matmul_w4(torch.ones((4, 64), device="cuda"), w).shape == (4, 0)


def test_values_that_are_not_finite_stay_in_their_row():
    torch = torch_cuda()
    rng = np.random.default_rng(4)
    codes, s, z, W, mag = make(rng, 1, 300, 50, 64, True, True, "float32")
    w = sg.w4_pack(codes[0], s[0], z[0], K=300, group=64)
    for rows in (1, 4, 9, 16, 40):
        for value in (float("nan"), float("inf"), float("-inf")):
            x = rng.integers(-4, 5, (rows, 300)).astype(np.float32)
            x[rows // 2, 137] = value
            got = run(x, w).double().cpu().numpy()
            want = np.delete(x, rows // 2, 0).astype(np.float64) @ W[0]
            assert not np.isfinite(got[rows // 2]).any()
            assert np.array_equal(np.delete(got, rows // 2, 0), want)
    # a NaN whose payload lies in its low bits
    x = np.ones((2, 300), np.float32)
    x.view(np.uint32)[0, 5] = 0x7F800001
    assert np.isnan(run(x, w)[0].cpu().numpy()).all()


def test_small_and_large_magnitudes():
    torch = torch_cuda()
    rng = np.random.default_rng(6)
    codes, s, z, W, mag = make(rng, 1, 256, 64, 128, True, False, "float32")
    w = sg.w4_pack(codes[0], s[0], z[0], K=256, group=128)
    x = (rng.standard_normal((8, 256)) * 10.0 ** np.array([-30, -20, -10, 0, 10, 20, 30, 34])[:, None]
         ).astype(np.float32)
    close(run(x, w), x.astype(np.float64) @ W[0], 256, np.abs(x.astype(np.float64)) @ mag[0], "w4")



@pytest.mark.parametrize("rows", [1, 5, 10, 16, 1600])
def test_magnitudes_next_to_the_smallest(rows):
    """Values whose last bits bf16 cannot hold: each may lose less than 2^-133, which scales of
    2^100 lift into sight (the sums themselves are far from the smallest numbers)."""
    torch = torch_cuda()
    rng = np.random.default_rng(rows)
    K, N, group = 256, 512, 64
    for zeros in (False, True):
        codes, s, z, W, mag = make(rng, 1, K, N, group, zeros, False, "float32")
        w = sg.w4_pack(codes[0], s[0] * 2.0**100, None if z is None else z[0], K=K, group=group)
        W, mag = W[0] * 2.0**100, mag[0] * 2.0**100
        for size in (1e-33, 1e-36, 1e-38, 1e-40):
            log(f"[gpu] w4 {rows} rows of {size}")
            x = (rng.standard_normal((rows, K)) * size).astype(np.float32)
            want = x.astype(np.float64) @ W
            off = np.abs(run(x, w).double().cpu().numpy() - want)
            limit = 1.01 * (3 * K + 8) * 2.0**-24 * (np.abs(x.astype(np.float64)) @ mag) + \
                1.01 * 2.0**-133 * mag.sum(0)
            assert (off <= limit).all(), (size, float((off / limit).max()))


def quantized(B, group, zeros, scale_type):
    """The formulas of the header in fp32: the matrix that the quantised B stands for."""
    torch = torch_cuda()
    out = np.zeros_like(B)
    for lo in range(0, B.shape[0], group):
        b = B[lo:lo + group]
        low, high = np.minimum(b.min(0), 0), np.maximum(b.max(0), 0)
        wide = (high - low) / np.float32(15) if zeros else np.maximum(-low, high) / np.float32(7)
        s = torch.from_numpy(wide).to(getattr(torch, scale_type)).float().numpy()
        safe = np.where(s > 0, s, np.float32(1))
        z = np.minimum(np.rint(-low / safe), np.float32(15)) if zeros else np.full_like(s, 8)
        q = np.minimum(np.maximum(np.rint(b / safe) + z, np.float32(0)), np.float32(15))
        out[lo:lo + group] = np.where(s > 0, s * (q - z), 0)
    return out


@pytest.mark.parametrize("K,N", [(1, 1), (128, 16), (100, 33), (257, 50), (1024, 64)])
@pytest.mark.parametrize("group", [32, 64, 128, 384])
def test_quantize_and_unpack(K, N, group):
    torch = torch_cuda()
    rng = np.random.default_rng(K + N)
    for zeros, scale_type in itertools.product((False, True), TYPES):
        B = rng.standard_normal((3, K, N)).astype(np.float32)
        B[1] = np.abs(B[1])
        B[2, :, : max(1, N // 2)] = 0.0
        wide = torch.full((3, K + 1, N + 3), float("nan"), device="cuda")
        wide[:, :K, :N] = torch.from_numpy(B).cuda()
        w = sg.w4_quantize(wide[:, :K, :N], group=group, zeros=zeros,
                           scale_dtype=getattr(torch, scale_type))
        got = sg.w4_unpack(w).cpu().numpy()
        for e in range(3):
            want = quantized(B[e], group, zeros, scale_type)
            # the device divides and rounds as the host does, but for ties that the
            # last bit of a quotient decides: those may take the neighbouring code
            step = np.abs(want - got[e])
            assert np.count_nonzero(step) <= max(2, want.size // 500)
        one = sg.w4_unpack(sg.w4_quantize(torch.from_numpy(B[0]).cuda(), group=group, zeros=zeros,
                                          scale_dtype=getattr(torch, scale_type))).cpu().numpy()
        assert np.array_equal(one, got[0])


@pytest.mark.parametrize("K,N,group", [(1, 1, 32), (33, 17, 32), (300, 40, 64), (513, 35, 128)])
def test_pack_and_unpack(K, N, group):
    torch = torch_cuda()
    rng = np.random.default_rng(K)
    for zeros, scale_type in itertools.product((False, True), TYPES):
        codes, s, z, W, _ = make(rng, 2, K, N, group, zeros, False, scale_type)
        w = sg.w4_pack(codes, s, z, K=K, group=group)
        # q - z and s are exact, so their product is rounded once
        assert np.array_equal(sg.w4_unpack(w).cpu().numpy(), W.astype(np.float32))


def test_quantized_product_next_to_the_full_one():
    """A user's way: quantise the matrix of an fp32 product, multiply, compare with
    the product of the matrix it stands for."""
    torch = torch_cuda()
    g = torch.Generator().manual_seed(2)
    A, B = torch.randn((7, 500), generator=g).cuda(), torch.randn((500, 300), generator=g).cuda()
    w = sg.w4_quantize(B, group=64, scale_dtype=torch.float16)
    C = sg.matmul_w4(A, w)
    full = sg.matmul(A, sg.w4_unpack(w))
    mag = A.abs().double() @ sg.w4_unpack(w).abs().double()
    # each side is within its own bound: (K + 4) and (3K + 8) roundings, q + z <= 23
    # times the smallest step where |q - z| may be 0, so in units of the group's scale
    scale = (B.abs().max() / 7).item()
    assert float((C - full).abs().max()) <= 2.0**-24 * (1.01 * 508 * 23 * scale * 3 *
                                                        float(A.abs().sum(1).max()) + float(mag.max()) * 504)


def test_packed_weights_beyond_32_bits():
    torch = torch_cuda()
    experts, K, N = 66, 8192, 16384
    codes = torch.full((experts, K // 2, N), 0x88, dtype=torch.uint8, device="cuda")
    codes[-1] = torch.randint(0, 256, (K // 2, N), dtype=torch.uint8, device="cuda")
    scales = torch.ones((experts, K // 128, N), dtype=torch.float16, device="cuda")
    w = sg.w4_pack(codes, scales, K=K, group=128)
    assert w.packed.numel() > 2**32
    one = sg.w4_pack(codes[-1].contiguous(), scales[-1].contiguous(), K=K, group=128)
    W = torch.stack((codes[-1] & 15, codes[-1] >> 4), 1).flatten(0, 1).double() - 8
    del codes
    for rows in (1, 4, 20, 70):
        x = torch.randint(-2, 3, (rows, K), device="cuda").float()
        off = torch.tensor([0] * experts + [rows], dtype=torch.int32, device="cuda")
        got = sg.matmul_w4(x, w, offsets=off)
        assert torch.equal(got.double(), x.double() @ W)
        assert torch.equal(got, sg.matmul_w4(x, one))
    out = torch.empty((1, K, N), device="cuda")
    assert sg.sgemm_f32_w4_unpack(1, N, K, 128, w.scale_type, 0,
                                  w.packed.data_ptr() + (experts - 1) * (w.packed.numel() // experts),
                                  w.packed.numel() // experts, out.data_ptr(), N, K * N,
                                  torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out[0].double(), W)


def test_calls_from_several_threads_and_streams():
    """Products with the same weights from four host threads, each on its own stream."""
    import threading
    torch = torch_cuda()
    rng = np.random.default_rng(21)
    codes, s, z, W, _ = make(rng, 1, 700, 300, 32, True, True, "float16")
    w = sg.w4_pack(codes[0], s[0], z[0], K=700, group=32)
    xs = [rng.integers(-4, 5, (rows, 700)).astype(np.float32) for rows in (1, 5, 17, 90)]
    dev = [torch.from_numpy(x).cuda() for x in xs]
    torch.cuda.synchronize()
    got = [[] for _ in xs]

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got[i].append(sg.matmul_w4(dev[i], w))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for x, results in zip(xs, got):
        assert len(results) == 20
        want = x.astype(np.float64) @ W[0]
        for c in results:
            assert np.array_equal(c.double().cpu().numpy(), want)


def test_graph_and_streams():
    torch = torch_cuda()
    rng = np.random.default_rng(9)
    codes, s, z, W, mag = make(rng, 6, 512, 200, 64, True, True, "float16")
    w = sg.w4_pack(codes, s, z, K=512, group=64)
    x = torch.empty((24, 512), device="cuda")
    off = torch.zeros(7, dtype=torch.int32, device="cuda")
    out = torch.empty((24, 200), device="cuda")
    one = sg.w4_pack(codes[0], s[0], z[0], K=512, group=64)
    single = torch.empty((24, 200), device="cuda")
    sg.matmul_w4(x, w, offsets=off, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.matmul_w4(x, w, offsets=off, out=out)
        sg.matmul_w4(x, one, out=single)
    for i in range(4):
        xi = rng.integers(-4, 5, (24, 512)).astype(np.float32)
        ends = [0] + sorted(rng.integers(0, 25, 5).tolist()) + [24]
        x.copy_(torch.from_numpy(xi))
        off.copy_(torch.tensor(ends, dtype=torch.int32))
        out.fill_(SENT)
        single.fill_(SENT)
        graph.replay()
        torch.cuda.synchronize()
        want = np.concatenate([xi[a:b].astype(np.float64) @ W[e]
                               for e, (a, b) in enumerate(zip(ends, ends[1:]))])
        assert np.array_equal(out.double().cpu().numpy(), want)
        assert np.array_equal(single.double().cpu().numpy(), xi.astype(np.float64) @ W[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = sg.matmul_w4(x, w, offsets=off, stream=side)
        side.synchronize()
        assert torch.equal(got, out)


def test_experts_layer_with_4_bit_weights():
    """Serving: rows to their experts, 4-bit products, rows back."""
    torch = torch_cuda()
    rng = np.random.default_rng(12)
    codes, s, z, W, _ = make(rng, 5, 96, 64, 32, False, True, "float16")
    w = sg.w4_pack(codes, s, z, K=96, group=32)
    for tokens in (1, 9, 40):
        ids = rng.integers(-1, 5, (tokens, 2)).astype(np.int32)
        x = rng.integers(-4, 5, (tokens, 96)).astype(np.float32)
        wt = 2.0 ** rng.integers(-2, 2, (tokens, 2)).astype(np.float32)
        r = sg.sort_by_expert(torch.from_numpy(ids).cuda(), 5)
        rows = sg.gather_rows(torch.from_numpy(x).cuda(), r)
        y = sg.matmul_w4(rows, w, offsets=r.offsets)
        got = sg.combine_rows(y, r, torch.from_numpy(wt).cuda()).double().cpu().numpy()
        want = np.zeros((tokens, 64))
        for t in range(tokens):
            for j in range(2):
                if ids[t, j] >= 0:
                    want[t] += wt[t, j] * (x[t].astype(np.float64) @ W[ids[t, j]])
        assert np.array_equal(got, want)


def test_refusals_of_the_torch_layer():
    torch = torch_cuda()
    dev = "cuda"
    codes = torch.zeros((32, 16), dtype=torch.uint8, device=dev)
    s = torch.ones((2, 16), device=dev)
    w = sg.w4_pack(codes, s, K=64, group=32)
    x = torch.zeros((4, 64), device=dev)
    stack = sg.w4_quantize(torch.ones((3, 64, 16), device=dev), group=32)
    off = torch.tensor([0, 1, 2, 4], dtype=torch.int32, device=dev)
    for f in (lambda: sg.w4_pack(codes, s, K=66, group=32), lambda: sg.w4_pack(codes, s, K=64, group=48),
              lambda: sg.w4_pack(codes, s[:1], K=64, group=32),
              lambda: sg.w4_pack(codes, s.double(), K=64, group=32),
              lambda: sg.w4_pack(codes.t(), s, K=64, group=32),
              lambda: sg.w4_pack(codes, s, s, K=64, group=32),
              lambda: sg.matmul_w4(x[:, :32], w), lambda: sg.matmul_w4(x, stack),
              lambda: sg.matmul_w4(x, stack, offsets=off[:3]),
              lambda: sg.matmul_w4(x, w, out=torch.zeros((4, 15), device=dev)),
              lambda: sg.matmul_w4(x.t().contiguous().t(), w),
              lambda: sg.matmul_w4(x.half(), w), lambda: sg.matmul_w4(x, stack, offsets=off.long()),
              lambda: sg.w4_quantize(torch.ones((3, 64, 16), device=dev).transpose(1, 2)),
              lambda: sg.w4_quantize(torch.ones((64, 16), device=dev), group=100)):
        with pytest.raises((ValueError, TypeError)):
            f()
    both = torch.zeros((8, 64), device=dev)
    with pytest.raises(sg.SgemmError):
        sg.matmul_w4(both[:4], w, out=both[2:6, :16])


@pytest.mark.parametrize("rows,N,K,group", [
    (1, 40, 3, 32), (1, 70, 300, 128), (5, 33, 129, 32), (9, 20, 200, 64), (16, 50, 260, 256),
    (40, 64, 300, 32), (70, 130, 140, 64), (1001, 2047, 140, 32), (2100, 2000, 200, 64),
    (513, 2900, 260, 128)])
def test_zero_points_above_15(rows, N, K, group):
    """Formats that keep a zero point of 16 (or any byte): taken as it is, in every kernel."""
    torch = torch_cuda()
    log(f"[gpu] w4 {rows} x {N} x {K} group {group}, zero points up to 255")
    rng = np.random.default_rng(rows + K)
    groups = -(-K // group)
    q = rng.integers(0, 16, (K + K % 2, N)).astype(np.uint8)
    x = rng.integers(-4, 5, (rows, K)).astype(np.float32)
    for z in (np.full((groups, N), 16, np.uint8), rng.integers(0, 256, (groups, N)).astype(np.uint8)):
        # |sum| <= 300 * 4 * 255 in steps of 1/2, at most 2^20 of them: exact in any order
        s = 2.0 ** rng.integers(-1, 1, (groups, N))
        w = sg.w4_pack(torch.from_numpy(q[0::2] | (q[1::2] << 4)).cuda(),
                       torch.from_numpy(s).to(torch.float16).cuda(), torch.from_numpy(z).cuda(),
                       K=K, group=group)
        W = np.repeat(s, group, 0)[:K] * (q[:K] - np.repeat(z, group, 0)[:K].astype(np.float64))
        assert np.array_equal(sg.w4_unpack(w).double().cpu().numpy(), W)
        got = sg.matmul_w4(torch.from_numpy(x).cuda(), w).double().cpu().numpy()
        assert np.array_equal(got, x.astype(np.float64) @ W)
