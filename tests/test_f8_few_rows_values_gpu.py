"""Rows that the product's own kernel puts into 8 bits (up to four), bit for bit the formula."""
import numpy as np
import pytest

import dense_fp32_matrix_f32_amd as sg
import f8_reference as ref
from gpu_helpers import log, torch_cuda
from test_f8_gpu import dtype_of, hard_rows, put, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("numbers", ["f32", "bf16"])
@pytest.mark.parametrize("few", [1, 3, 4])
@pytest.mark.parametrize("K", [1, 3, 17, 127, 128, 130, 300, 1100])
def test_few_rows_are_the_formula(K, few, numbers, kind):
    """With the identity for weights a product is the rows themselves."""
    torch = torch_cuda()
    log(f"[gpu] f8 {few} rows x {K} {numbers} {kind}")
    # no workspace: there is no kernel that puts the rows into 8 bits before
    assert sg.sgemm_f32_f8_workspace_size(few, K, K, 1, 0) == 0
    eye = torch.eye(K, device="cuda").to(dtype_of("e4m3"))
    ones = torch.ones((-(-K // 128),) * 2, device="cuda")
    a, x = put(hard_rows(K), pad=few, offset=few, kind=numbers)
    want = ref.rows(x, kind)
    # fp32's largest number becomes 2^128 in 8 bits, which is infinite in 32: times zeros NaN
    huge = (np.abs(want) >= 2.0**128).any(axis=1)
    assert huge.sum() == (1 if numbers == "f32" else 0)
    want[huge] = np.nan if K > 1 else np.inf
    # an infinite value (hard_rows has one for 1100) is NaN in 8 bits, and so is its row of a product
    want[~np.isfinite(x).all(axis=1)] = np.nan
    for scales in (ones, ones.to(dtype_of("e8m0"))):
        w = sg.f8_pack(eye, scales)
        same(torch.cat([sg.matmul_f8(part, w, dtype=dtype_of(kind)) for part in a.split(few)]), want)
    # and by expert, as many rows for each of two on average
    n = a.shape[0] // few // 2 * 2 * few
    w = sg.f8_pack(eye[None].repeat(2, 1, 1), ones[None].repeat(2, 1, 1))
    off = torch.tensor([0, few, 2 * few], dtype=torch.int32, device="cuda")
    assert sg.sgemm_f32_f8_workspace_size(2 * few, K, K, 2, 1) == 0
    same(torch.cat([sg.matmul_f8(part, w, offsets=off, dtype=dtype_of(kind)) for part in a[:n].split(2 * few)]), want[:n])
