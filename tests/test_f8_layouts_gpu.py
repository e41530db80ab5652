"""Codes and scales are packed in one layout: both row-major, or both transposed views."""
import pytest

import dense_fp32_matrix_f32_amd as sg
from gpu_helpers import log, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stacked", [False, True])
def test_scales_are_in_the_layout_of_the_codes(stacked):
    torch = torch_cuda()
    log(f"[gpu] f8 pack layouts, stacked {stacked}")
    K, N = 300, 200
    lead = (3,) if stacked else ()
    codes = torch.randint(-8, 9, lead + (N, K), device="cuda").float().to(torch.float8_e4m3fn)
    scales = torch.rand(lead + (2, 3), device="cuda")
    tc, ts = codes.transpose(-1, -2), scales.transpose(-1, -2)
    rc, rs = tc.contiguous(), ts.contiguous()
    want = sg.f8_unpack(sg.f8_pack(rc, rs))
    assert torch.equal(sg.f8_unpack(sg.f8_pack(tc, ts)), want)
    with pytest.raises(ValueError, match="transposed view of a contiguous array"):
        sg.f8_pack(tc, rs)
    with pytest.raises(ValueError, match="contiguous, as codes is row-major"):
        sg.f8_pack(rc, ts)
