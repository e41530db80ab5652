"""A layer of experts with matrices in 8 bits whose rows are near the end of fp32's range, with scales
that bring the results back into it (tolerance: that of test_layer_gpu.py)."""
import numpy as np
import pytest

import dense_fp32_matrix_f32_amd as sg
import f8_reference as ref
from gpu_helpers import log, torch_cuda
from test_layer_gpu import reference

pytestmark = pytest.mark.gpu


def stack(rng, experts, K, N, low, high, zero=None):
    """(a stack, the matrices in 64 bits, their sizes); `zero`: a block of k with a scale of zero."""
    torch = torch_cuda()
    codes = torch.from_numpy(np.clip(rng.standard_normal((experts, K, N)) * 100, -448, 448).astype(np.float32)
                             ).to(torch.float8_e4m3fn)
    s = rng.uniform(low, high, (experts, -(-K // 128), -(-N // 128))).astype(np.float32)
    s *= rng.choice([-1, 1], s.shape).astype(np.float32)
    if zero is not None:
        s[:, zero] = 0
    m = ref.scaled(codes.double().numpy(), s.astype(np.float64))
    return sg.f8_pack(codes.cuda(), torch.from_numpy(s).cuda()), m, np.abs(m)


def layer(x, ids, weights, up, down, gate=None):
    torch = torch_cuda()
    t = [torch.from_numpy(a).cuda() for a in (x, ids, weights)]
    return sg.expert_layer(*t, up[0], down[0], gate=gate[0] if gate else None, act="relu")


SHAPES = [(1, 1, 1), (1, 4, 8), (3, 2, 8), (20, 2, 3), (64, 3, 4)]


@pytest.mark.parametrize("tokens,top,experts", SHAPES)
@pytest.mark.parametrize("width,hidden", [(300, 390), (2, 300), (260, 3)])
@pytest.mark.parametrize("size", [1e33, 1e35, 1e36])
def test_large_rows(tokens, top, experts, width, hidden, size):
    rng = np.random.default_rng(tokens + width)
    log(f"[gpu] layer of {tokens} rows of {size}, {width} x {hidden}")
    up, down = stack(rng, experts, width, hidden, 1e-5, 1e-4), stack(rng, experts, hidden, width, 1e-5, 1e-4)
    x = (size * rng.standard_normal((tokens, width))).astype(np.float32)
    ids = np.stack([rng.permutation(experts)[:top] for _ in range(tokens)]).astype(np.int32)
    weights = rng.uniform(-1, 1, (tokens, top)).astype(np.float32)
    got = layer(x, ids, weights, up, down).double().cpu().numpy()
    want, off = reference(x.astype(np.float64), ids, weights, up, None, down, "relu")
    assert np.abs(want).max() < 1e38
    bad = ~(np.abs(got - want) <= off)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, {int((~np.isfinite(got)).sum())} no numbers"


@pytest.mark.parametrize("tokens,top,experts", SHAPES)
@pytest.mark.parametrize("gated", [False, True])
def test_scales_of_zero_next_to_the_largest_rows(tokens, top, experts, gated):
    """A block of either matrix with a scale of zero adds nothing, however large the rows are there."""
    torch = torch_cuda()
    rng = np.random.default_rng(tokens)
    log(f"[gpu] layer of {tokens} rows next to scales of zero, gated {gated}")
    width, hidden = 384, 300
    up = stack(rng, experts, width, hidden, 1e-3, 1e-2, zero=1)
    gate = stack(rng, experts, width, hidden, 1e-3, 1e-2, zero=1) if gated else None
    down = stack(rng, experts, hidden, width, 1e-3, 1e-2, zero=0)
    x = rng.standard_normal((tokens, width)).astype(np.float32)
    x[:, 128:256] = rng.uniform(-1, 1, (tokens, 128)) * 2.0**127
    ids = np.stack([rng.permutation(experts)[:top] for _ in range(tokens)]).astype(np.int32)
    weights = rng.uniform(-1, 1, (tokens, top)).astype(np.float32)
    got = layer(x, ids, weights, up, down, gate)
    x[:, 128:256] = 0
    want = layer(x, ids, weights, up, down, gate)
    assert bool(want.abs().max() > 0) and torch.equal(got, want)
