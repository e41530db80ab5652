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
