"""A layer with as many choices of a token and tokens of a round as it takes, for so many experts that
the second kernel's tables leave its LDS no room for the sums of four strips of columns (from 411
experts on), and just before that (tolerance: that of test_layer_gpu.py)."""
import numpy as np
import pytest

from gpu_helpers import log
from test_layer_gpu import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,form", [("f8", 0), ("f8", 1), ("w4", 0), ("w4", 1), ("w4", 2)])
@pytest.mark.parametrize("experts", [409, 410, 411, 500, 1000, 2048, 3000])
def test_all_choices_of_all_tokens(kind, form, experts):
    rng = np.random.default_rng(experts + form)
    log(f"[gpu] layer of 64 tokens, 32 of {experts}")
    check(rng, 64, 32, experts, 20, 70, kind, "silu", True, form, dropped=0.05)
    check(rng, 64, 32, experts, 130, 20, kind, "relu", False, form, dropped=0.0)
