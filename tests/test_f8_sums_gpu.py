"""Sums of the products in 8 bits are kept in 32 bits, whatever the result's type and the
number of rows.

Rows and weights of whole numbers up to 256 whose largest products (2^16) cancel: every sum of
some of an element's terms is a multiple of 1/2 below 2^22, so fp32 holds it in any order, and a
result is the formula's, rounded once.  Sums that keep 14 bits below their largest term lose the
small products next to the large ones."""
import numpy as np
import pytest

import dense_fp32_matrix_f32_amd as sg
import f8_reference as ref
from gpu_helpers import log, torch_cuda
from test_f8_gpu import dtype_of, put, rounded, run, same

pytestmark = pytest.mark.gpu


def cancelling(rng, rows, K, N, experts):
    """(x, codes): of each eight k the first two are large and cancel, the others 0 to 3."""
    x = rng.integers(0, 4, (rows, K)).astype(np.float32)
    w = rng.integers(-3, 4, (experts, K, N)).astype(np.float32)
    x[:, 0::8] = x[:, 1::8] = 256
    big = 256 * rng.choice([-1.0, 1.0], (experts, len(range(0, K, 8)), N))
    w[:, 0::8] = big
    w[:, 1::8] = -big
    return x, w


@pytest.mark.parametrize("rows,N,K", [(3, 70, 128), (20, 130, 256), (200, 130, 256), (300, 100, 128), (300, 1030, 256),
                                      (1200, 4100, 256), (4000, 8200, 128)])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_large_terms_that_cancel(rows, N, K, kind):
    torch = torch_cuda()
    rng = np.random.default_rng(rows + N)
    x, codes = cancelling(rng, rows, K, N, 1)
    for scale in ("f32", "e8m0"):
        s = rng.choice([0.5, 1.0, 1.5] if scale == "f32" else [0.5, 1.0], (-(-K // 128), -(-N // 128))).astype(np.float32)
        w = sg.f8_pack(torch.from_numpy(codes[0]).cuda().to(dtype_of("e4m3")),
                       torch.from_numpy(s).cuda().to(torch.float32 if scale == "f32" else dtype_of("e8m0")))
        want = x.astype(np.float64) @ ref.scaled(codes[0].astype(np.float64), s.astype(np.float64))
        assert np.abs(want).max() < 2.0**13
        for result in ("bf16", "f32"):
            log(f"[gpu] f8 sums {rows} x {N} x {K} {kind} scales {scale} {result}")
            a, _ = put(x, kind="bf16" if result == "bf16" else "f32")
            same(run(a, w, result, dtype=dtype_of(kind)), rounded(want, result).double().numpy())


@pytest.mark.parametrize("rows,N,experts", [(30, 130, 4), (1500, 130, 4), (3000, 2100, 8)])
def test_large_terms_that_cancel_by_expert(rows, N, experts):
    torch = torch_cuda()
    rng = np.random.default_rng(rows)
    K = 256
    x, codes = cancelling(rng, rows, K, N, experts)
    off = np.sort(np.concatenate([[0, rows], rng.integers(0, rows, experts - 1)])).astype(np.int32)
    s = rng.choice([0.5, 1.0, 1.5], (experts, 2, -(-N // 128))).astype(np.float32)
    w = sg.f8_pack(torch.from_numpy(codes).cuda().to(dtype_of("e4m3")), torch.from_numpy(s).cuda())
    W = ref.scaled(codes.astype(np.float64), s.astype(np.float64))
    want = np.concatenate([x[lo:hi].astype(np.float64) @ W[e] for e, (lo, hi) in enumerate(zip(off, off[1:]))])
    for result in ("bf16", "f32"):
        log(f"[gpu] f8 sums by expert {experts}: {rows} x {N} {result}")
        a, _ = put(x)
        same(run(a, w, result, offsets=torch.from_numpy(off).cuda()), rounded(want, result).double().numpy())
