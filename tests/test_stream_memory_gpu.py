"""Results of calls on a stream that is passed in, next to work that still runs on the
current stream over memory of the results' size that has just been freed."""
import numpy as np
import pytest

import dense_fp32_matrix_f32_amd as sg
from gpu_helpers import log, torch_cuda

pytestmark = pytest.mark.gpu


def tensors(result):
    """The tensors of a result: itself, packed weights, or a tuple of these."""
    if isinstance(result, sg.W4Weights):
        return [result.packed]
    if isinstance(result, tuple):
        return [t for r in result for t in tensors(r)]
    return [] if result is None else [result]


def check(call):
    """call(stream) on a side stream, while the current stream still has to read blocks
    that were freed there and have the sizes of the results: the call may neither
    change what is read nor give other results."""
    torch = torch_cuda()
    want = [t.clone() for t in tensors(call(None))]
    side = torch.cuda.Stream()
    big = torch.ones((4096, 4096), device="cuda")
    slow = torch.empty_like(big)
    torch.cuda.synchronize()
    for _ in range(2):
        # three blocks for each result, and as many for a workspace
        freed = [torch.full_like(t, 3) for t in want for _ in range(3)]
        read = [torch.zeros_like(t) for t in freed]
        torch.cuda.synchronize()
        for _ in range(4):
            torch.mm(big, big, out=slow)  # a millisecond each
        for r, t in zip(read, freed):
            r.copy_(t)
        places = {t.data_ptr() for t in freed if t.numel()}
        del freed, t
        got = tensors(call(side))
        mine = {t.data_ptr() for t in got if t.numel()}
        side.synchronize()
        torch.cuda.synchronize()
        assert not places & mine, "memory that the current stream still reads was written"
        for r in read:
            assert r.eq(3).all()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del got, read


def routed():
    torch = torch_cuda()
    rng = np.random.default_rng(5)
    ids = torch.from_numpy(rng.integers(0, 8, (3000, 3)).astype(np.int32)).cuda()
    x = torch.from_numpy(rng.integers(-4, 5, (3000, 72)).astype(np.float32)).cuda()
    y = torch.from_numpy(rng.integers(-4, 5, (9000, 72)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.integers(1, 4, (3000, 3)).astype(np.float32)).cuda()
    B = torch.from_numpy(rng.integers(-4, 5, (8, 72, 72)).astype(np.float32)).cuda()
    return sg.sort_by_expert(ids, 8), ids, x, y, w, B


@pytest.mark.parametrize("name", ["sort", "gather", "combine", "combine_grad", "grouped",
                                  "grouped_ta"])
def test_rows_and_products_by_expert(name):
    log(f"[gpu] {name} on another stream over freed memory")
    r, ids, x, y, w, B = routed()
    check({"sort": lambda s: sg.sort_by_expert(ids, 8, stream=s),
           "gather": lambda s: sg.gather_rows(x, r, stream=s),
           "combine": lambda s: sg.combine_rows(y, r, w, stream=s),
           "combine_grad": lambda s: sg.combine_rows_grad(x, y, r, w, stream=s),
           "grouped": lambda s: sg.grouped_matmul(y, B, r.offsets, stream=s),
           "grouped_ta": lambda s: sg.grouped_matmul_ta(y, y, r.offsets, stream=s)}[name])


@pytest.mark.parametrize("name", ["pack", "quantize", "unpack", "product", "by expert"])
def test_4_bit_weights(name):
    torch = torch_cuda()
    log(f"[gpu] 4-bit {name} on another stream over freed memory")
    r, _, _, y, _, _ = routed()
    rng = np.random.default_rng(6)
    # sizes without padding, so that every byte of the packed array is written
    codes = torch.from_numpy(rng.integers(0, 256, (8, 64, 64)).astype(np.uint8)).cuda()
    scales = torch.ones((8, 4, 64), device="cuda")
    stack = sg.w4_pack(codes, scales, K=128, group=32)
    one = sg.w4_pack(codes[0], scales[0], K=128, group=32)
    full = sg.w4_unpack(stack)
    a = torch.from_numpy(rng.integers(-4, 5, (9000, 128)).astype(np.float32)).cuda()
    check({"pack": lambda s: sg.w4_pack(codes, scales, K=128, group=32, stream=s),
           "quantize": lambda s: sg.w4_quantize(full, group=32, stream=s),
           "unpack": lambda s: sg.w4_unpack(stack, stream=s),
           "product": lambda s: sg.matmul_w4(a, one, stream=s),
           "by expert": lambda s: sg.matmul_w4(a, stack, offsets=r.offsets, stream=s)}[name])


@pytest.mark.parametrize("M,N,K,workspace", [(300, 257, 131, None), (128, 96, 30000, "auto")])
def test_matmul(M, N, K, workspace):
    torch = torch_cuda()
    log(f"[gpu] matmul {M}x{N}x{K} on another stream over freed memory")
    rng = np.random.default_rng(7)
    a, b = (torch.from_numpy(rng.integers(-4, 5, s).astype(np.float32)).cuda()
            for s in ((M, K), (K, N)))
    if workspace:
        assert sg.sgemm_f32_workspace_size(0, 0, M, N, K) > 0
    check(lambda s: sg.matmul(a, b, workspace=workspace, stream=s))


@pytest.mark.parametrize("null", [False, True])
def test_a_stream_known_by_its_handle(null):
    """An object that only holds a stream's handle will do, the null stream's included."""
    torch = torch_cuda()
    side = torch.cuda.Stream()
    r, ids, x, _, _, _ = routed()

    class Handle:
        cuda_stream = 0 if null else side.cuda_stream

    want = sg.gather_rows(x, r)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = sg.gather_rows(x, r, stream=Handle())
    (torch.cuda.default_stream() if null else side).synchronize()
    assert torch.equal(got, want)


def test_a_stream_of_another_gpu_is_refused():
    torch = torch_cuda()
    r, ids, x, y, w, B = routed()
    one = sg.w4_quantize(B[0], group=32)

    class Other:
        device = torch.device("cuda", torch.cuda.current_device() + 1)
        cuda_stream = torch.cuda.Stream().cuda_stream

    out = torch.empty_like(y)
    for f in (lambda s: sg.sort_by_expert(ids, 8, stream=s), lambda s: sg.gather_rows(x, r, stream=s),
              lambda s: sg.gather_rows(x, r, out=out, stream=s),
              lambda s: sg.combine_rows(y, r, stream=s),
              lambda s: sg.combine_rows_grad(x, y, r, w, stream=s),
              lambda s: sg.grouped_matmul(y, B, r.offsets, out=out, stream=s),
              lambda s: sg.grouped_matmul_ta(y, y, r.offsets, stream=s),
              lambda s: sg.w4_quantize(B, group=32, stream=s), lambda s: sg.w4_unpack(one, stream=s),
              lambda s: sg.matmul_w4(y, one, out=out, stream=s),
              lambda s: sg.matmul(y, B[0], out=out, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            f(Other())


def test_another_stream_inside_a_capture():
    """Calls on a stream that a capture has forked to: replayed on new inputs, with eager
    work between the replays."""
    torch = torch_cuda()
    r, ids, x, _, w, B = routed()
    side, out = torch.cuda.Stream(), torch.empty_like(x)

    def layer(stream):
        r = sg.sort_by_expert(ids, 8, stream=stream)
        h = sg.grouped_matmul(sg.gather_rows(x, r, stream=stream), B, r.offsets, stream=stream)
        return sg.combine_rows(h, r, w, stream=stream), sg.matmul(x, B[0], stream=stream)

    layer(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = layer(side)
        torch.cuda.current_stream().wait_stream(side)
        out.copy_(got[0])
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids.copy_(torch.randint(-1, 8, ids.shape, generator=g, device="cuda"))
        x.copy_(torch.randint(-4, 5, x.shape, generator=g, device="cuda"))
        want = layer(None)
        torch.cuda.synchronize()
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*got, out), (*want, want[0])):
            assert torch.equal(a, b)
