"""Products in 8 bits of rows near the end of fp32's range, with fp32 scales that bring the
result back into it.

Tolerance: as for any product with an fp32 sum, 1.01 * (K + K / 128 + 16) * 2^-24 of the sum of
the terms without signs, and with a bf16 result 2^-8 of the value for its rounding."""
import numpy as np
import pytest

import dense_fp32_matrix_f32_amd as sg
import f8_reference as ref
from gpu_helpers import log, torch_cuda
from test_f8_gpu import dtype_of, run, same

pytestmark = pytest.mark.gpu

ROWS = [1, 4, 20, 200, 300, 1200]


def codes_of(rng, K, N):
    torch = torch_cuda()
    return torch.from_numpy(np.clip(rng.standard_normal((K, N)) * 100, -448, 448).astype(np.float32)).to(dtype_of("e4m3"))


def check(x, codes, s, result, by_expert=False):
    torch = torch_cuda()
    if by_expert:
        w = sg.f8_pack(codes[None].cuda(), torch.from_numpy(s)[None].cuda())
        more = dict(offsets=torch.tensor([0, len(x)], dtype=torch.int32, device="cuda"))
    else:
        w, more = sg.f8_pack(codes.cuda(), torch.from_numpy(s).cuda()), {}
    got = run(torch.from_numpy(x).cuda(), w, result, **more).double().cpu().numpy()
    K = x.shape[1]
    x8, W = ref.rows(x.astype(np.float64)), ref.scaled(codes.double().numpy(), s.astype(np.float64))
    want, mag = x8 @ W, np.abs(x8) @ np.abs(W)
    assert mag.max() < 3.3e38
    limit = 1.01 * (K + K / 128 + 16) * 2.0**-24 * mag + 1e-37
    if result == "bf16":
        limit = limit + 2.0**-8 * (np.abs(want) + limit)
    bad = ~(np.abs(got - want) <= limit)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, {int((~np.isfinite(got)).sum())} no numbers"


@pytest.mark.parametrize("result", ["f32", "bf16"])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("size", [1e33, 1e34, 1e35, 1e36])
def test_large_rows(rows, size, result):
    rng = np.random.default_rng(rows)
    K, N = 384, 300
    log(f"[gpu] f8 rows of {size}, {rows} rows {result}")
    x = (size * rng.standard_normal((rows, K))).astype(np.float32)
    s = rng.uniform(1e-4, 1e-3, (3, 3)).astype(np.float32) * rng.choice([-1, 1], (3, 3)).astype(np.float32)
    codes = codes_of(rng, K, N)
    check(x, codes, s, result)
    check(x, codes, s, result, by_expert=True)


@pytest.mark.parametrize("result", ["f32", "bf16"])
@pytest.mark.parametrize("rows", ROWS)
def test_one_large_value(rows, result):
    """1e35 times a code of 448 with a scale of 1e-4 is 4.5e33."""
    torch = torch_cuda()
    log(f"[gpu] f8 one large value, {rows} rows {result}")
    x = np.full((rows, 128), 1e35, np.float32)
    codes = torch.full((128, 64), 448.0).to(dtype_of("e4m3"))
    check(x, codes, np.full((1, 1), 1e-4, np.float32), result)


@pytest.mark.parametrize("result", ["f32", "bf16"])
@pytest.mark.parametrize("rows", ROWS)
def test_scales_of_zero_next_to_the_largest_rows(rows, result):
    """A block of weights with a scale of zero adds nothing next to rows of up to 2^127."""
    torch = torch_cuda()
    rng = np.random.default_rng(rows)
    log(f"[gpu] f8 scales of zero, largest rows, {rows} rows {result}")
    K, N = 384, 300
    codes = codes_of(rng, K, N)
    s = rng.uniform(0.01, 1, (3, 3)).astype(np.float32)
    s[1] = 0
    x = rng.standard_normal((rows, K)).astype(np.float32)
    x[:, 128:256] = rng.uniform(-1, 1, (rows, 128)) * 2.0**127
    w = sg.f8_pack(codes.cuda(), torch.from_numpy(s).cuda())
    got = sg.matmul_f8(torch.from_numpy(x).cuda(), w, out_dtype=dtype_of(result))
    x[:, 128:256] = 0
    want = sg.matmul_f8(torch.from_numpy(x).cuda(), w, out_dtype=dtype_of(result))
    assert bool(want.abs().max() > 0) and torch.equal(got, want)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("power", [-130, -127, -126, -100, 60, 100])
def test_scales_near_the_ends(rows, power):
    """Powers of two as fp32 scales (below 2^-126 they have no leading bit), with rows that bring the
    result near one: whole codes from 1 on, exact in any order, so bit for bit."""
    torch = torch_cuda()
    rng = np.random.default_rng(rows)
    log(f"[gpu] f8 scale 2^{power}, {rows} rows")
    codes = rng.integers(1, 9, (256, 70)).astype(np.float64)
    x = (rng.integers(-4, 5, (rows, 256)) * 2.0 ** min(-power, 120)).astype(np.float32)
    s = np.full((2, 1), 2.0**power, np.float32)
    w = sg.f8_pack(torch.from_numpy(codes).cuda().to(dtype_of("e4m3")), torch.from_numpy(s).cuda())
    same(sg.matmul_f8(torch.from_numpy(x).cuda(), w), x.astype(np.float64) @ (codes * 2.0**power))
