"""Values of the 4-bit operators at their limits, and each element against its own bound.

Tolerance of a product, as derived in test_w4_gpu.py: with |terms| = |x| * s * (q + z)
the result is within 1.01 * (3K + 8) * 2^-24 * sum |terms| in any order."""
import numpy as np
import pytest

import dense_fp32_matrix_f32_amd as sg
from gpu_helpers import log, torch_cuda

pytestmark = pytest.mark.gpu


def within(got, want, limit, what):
    """Every element finite and no further than its limit from `want`."""
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: {np.count_nonzero(~np.isfinite(got))} not finite"
    worst = float((np.abs(got - want) / np.maximum(limit, 1e-300)).max())
    assert worst <= 1.0, f"{what}: the worst element is off by {worst:.3g} of its bound"


@pytest.mark.parametrize("rows", [1, 4, 9, 16, 60, 1000])
@pytest.mark.parametrize("group", [32, 64, 128, 384])
def test_largest_values_that_cannot_overflow(rows, group):
    """Rows of one sign at the limit that the header states, all codes 15: the sums of a
    group come within 4% of the largest fp32 number."""
    torch = torch_cuda()
    log(f"[gpu] w4 {rows} rows, group {group}, at the largest values")
    N, K = 300 if rows < 1000 else 2100, 400
    rng = np.random.default_rng(group)
    for z, top in [(None, 2.2e37), (0, 2.2e37), (15, 2.2e37), (255, 1.3e36)]:
        a = np.float32(top) / np.float32(min(group, 128)) * (1 - 2.0**-20)
        x = np.full((rows, K), a, np.float32)
        x[1::2] *= -1
        x[2::3] *= np.where(rng.random((1, K)) < 0.5, -1, 1)
        q = np.full((K, N), 15, np.uint8)
        q[:, 1::2] = rng.integers(0, 16, (K, N // 2))
        groups = -(-K // group)
        w = sg.w4_pack(torch.from_numpy(q[0::2] | (q[1::2] << 4)).cuda(),
                       torch.full((groups, N), 2.0**-12, device="cuda"),
                       None if z is None else torch.full((groups, N), z, dtype=torch.uint8,
                                                         device="cuda"), K=K, group=group)
        zero = 8 if z is None else z
        want = x.astype(np.float64) @ ((q.astype(np.float64) - zero) * 2.0**-12)
        mag = np.abs(x.astype(np.float64)) @ ((q.astype(np.float64) + zero) * 2.0**-12)
        within(sg.matmul_w4(torch.from_numpy(x).cuda(), w), want,
               1.01 * (3 * K + 8) * 2.0**-24 * mag, f"z {z}")


def quantized(B, group, zeros, scale_dtype):
    """The header's formulas in fp32, one operation after the other: (scales, zero points,
    codes), a row for each k."""
    torch = torch_cuda()
    s, z, q = (np.zeros(B.shape, np.float32) for _ in range(3))
    for lo in range(0, B.shape[0], group):
        at = slice(lo, lo + group)
        b = B[at]
        low, high = np.minimum(b.min(0), np.float32(0)), np.maximum(b.max(0), np.float32(0))
        wide = (high - low) / np.float32(15) if zeros else np.maximum(-low, high) / np.float32(7)
        one = torch.from_numpy(wide).to(scale_dtype).float().numpy()
        safe = np.where(one > 0, one, np.float32(1))
        z[at] = np.where(one > 0, np.minimum(np.rint(-low / safe), np.float32(15)), 8) if zeros else 8
        s[at] = one
        q[at] = np.where(one > 0, np.clip(np.rint(b / safe) + z[at], 0, 15), z[at])
    return s, z, q


@pytest.mark.parametrize("K,N", [(1, 1), (31, 17), (128, 16), (100, 33), (257, 50), (1024, 64)])
@pytest.mark.parametrize("group", [32, 64, 128, 384, 2048])
@pytest.mark.parametrize("values", ["normal", "positive", "negative", "ties", "sizes"])
def test_quantize_to_the_last_code(K, N, group, values):
    """Division, rint and the rounding of the scale are IEEE on both sides, so every
    value equals the formula's, at ties too."""
    torch = torch_cuda()
    log(f"[gpu] w4 quantize {K} x {N} group {group}, {values}")
    rng = np.random.default_rng(K + N + group)
    for zeros in (False, True):
        for scale_dtype in (torch.float32, torch.float16, torch.bfloat16):
            B = rng.standard_normal((2, K, N)).astype(np.float32)
            if values == "positive":
                B = np.abs(B)
            elif values == "negative":
                B = -np.abs(B)
            elif values == "ties":  # halves of a step of 1/4 (with a 7/4 in each column)
                B = (rng.integers(-14, 15, (2, K, N)) / np.float32(8)).astype(np.float32)
                B[:, ::min(group, 32)] = 1.75
            elif values == "sizes":
                B *= np.float32(2) ** rng.integers(-12, 12, (2, K, N)).astype(np.float32)
                B[:, :, ::3] = 0
            w = sg.w4_quantize(torch.from_numpy(B).cuda(), group=group, zeros=zeros,
                               scale_dtype=scale_dtype)
            got = sg.w4_unpack(w).cpu().numpy()
            for e in range(2):
                s, z, q = quantized(B[e], group, zeros, scale_dtype)
                assert np.array_equal(got[e], s * (q - z))
                # what the formula is for: no value further than half a step from its code
                # (and what the rounded scale leaves out at the ends)
                inside = np.rint(B[e] / np.where(s > 0, s, 1)) + z == q
                step = np.abs(got[e].astype(np.float64) - B[e])[inside & (s > 0)]
                assert (step <= s[inside & (s > 0)] * (0.5 + 2.0**-18)).all()


@pytest.mark.parametrize("rows", [1, 2, 5, 7, 16, 33, 90, 700])
@pytest.mark.parametrize("zeros,scale", [(False, "float16"), (True, "bfloat16"), (True, "float32")])
def test_each_element_of_a_product_with_a_quantised_matrix(rows, zeros, scale):
    """A user's way: quantise a matrix, multiply, compare with the product of the matrix
    it stands for, each element with the bound of its own terms."""
    torch = torch_cuda()
    log(f"[gpu] w4 product with a quantised matrix, {rows} rows")
    rng = np.random.default_rng(rows)
    K, N, group = 500, 2050, 64
    x = (rng.standard_normal((rows, K)) * 10.0 ** rng.integers(-3, 4, (rows, 1))).astype(np.float32)
    B = (rng.standard_normal((K, N)) * 10.0 ** rng.integers(-3, 4, (1, N))).astype(np.float32)
    w = sg.w4_quantize(torch.from_numpy(B).cuda(), group=group, zeros=zeros,
                       scale_dtype=getattr(torch, scale))
    s, z, q = (t.astype(np.float64) for t in quantized(B, group, zeros, getattr(torch, scale)))
    X = x.astype(np.float64)
    within(sg.matmul_w4(torch.from_numpy(x).cuda(), w), X @ (s * (q - z)),
           1.01 * (3 * K + 8) * 2.0**-24 * (np.abs(X) @ (s * (q + z))), "product")
