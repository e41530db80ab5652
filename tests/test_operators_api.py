"""Host-side checks of the operators around the product (4-bit weights, rows by
expert, the experts' products): refusals, empty calls, packed sizes and the torch
layer's checks of its arguments.  No kernel is launched."""
import pytest

import dense_fp32_matrix_f32_amd as sg
from dense_fp32_matrix_f32_amd import _binding

INVALID = _binding.HIP_ERROR_INVALID_VALUE

# Fake, well-separated "device" addresses: validation only looks at the numbers.
A, B, C, D, E, F, G = ((i + 1) << 36 for i in range(7))
MAX = 2**31 - 1


def _refused(entry, base, bad, order):
    args = {**base, **bad}
    st = getattr(sg, entry)(*[args[k] for k in order])
    assert st == INVALID, (entry, bad, st)


SORT = dict(tokens=8, top=2, experts=4, ids=A, ldids=2, offsets=B, order=C, position=D, ws=E,
            ws_bytes=1 << 20)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(top=-1), dict(experts=-1), dict(ldids=1), dict(ids=0), dict(offsets=0),
    dict(order=0), dict(position=0), dict(tokens=MAX, top=2), dict(experts=MAX),
    dict(order=A + 8), dict(position=C + 60), dict(offsets=D + 4), dict(offsets=A + 16)])
def test_sort_refuses(bad):
    _refused("sgemm_f32_route_sort", SORT, bad, SORT)


def test_sort_checks_its_workspace():
    # sizes at which a workspace is needed, if any are
    for tokens, top, experts in [(8, 2, 4), (32768, 8, 256), (1 << 20, 4, 64)]:
        need = sg.sgemm_f32_route_workspace_size(tokens, top, experts)
        if need == 0:
            continue
        big = {**SORT, "tokens": tokens, "top": top, "ldids": top, "experts": experts,
               "ws_bytes": need}
        for bad in [dict(ws=0), dict(ws_bytes=need - 1), dict(ws=E + 4), dict(ws=A + 16),
                    dict(ws=C + 16)]:
            _refused("sgemm_f32_route_sort", big, bad, SORT)
    assert sg.sgemm_f32_route_workspace_size(-1, 2, 4) == 0
    assert sg.sgemm_f32_route_workspace_size(MAX, 2, 4) == 0


GATHER = dict(tokens=8, top=2, width=16, position=A, x=B, ldx=16, rows=C, ldrows=16)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(top=-1), dict(width=-1), dict(ldx=15), dict(ldrows=15), dict(position=0),
    dict(x=0), dict(rows=0), dict(tokens=MAX, top=3), dict(rows=B + 64), dict(rows=A + 4)])
def test_gather_refuses(bad):
    _refused("sgemm_f32_route_gather", GATHER, bad, GATHER)


COMBINE = dict(tokens=8, top=2, width=16, position=A, weights=B, ldw=2, rows=C, ldrows=16, out=D,
               ldout=16)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(top=-1), dict(width=-1), dict(ldw=1), dict(ldrows=15), dict(ldout=15),
    dict(position=0), dict(rows=0), dict(out=0), dict(out=C + 64), dict(out=B + 4),
    dict(out=A + 4)])
def test_combine_refuses(bad):
    _refused("sgemm_f32_route_combine", COMBINE, bad, COMBINE)


GRAD = dict(tokens=8, top=2, width=16, position=A, weights=B, ldw=2, rows=C, ldrows=16, dout=D,
            lddout=16, drows=E, lddrows=16, dweights=F)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(top=-1), dict(width=-1), dict(ldw=1), dict(ldrows=15), dict(lddout=15),
    dict(lddrows=15), dict(position=0), dict(rows=0), dict(dout=0), dict(drows=C + 64),
    dict(drows=D + 64), dict(dweights=E + 4), dict(dweights=B + 4), dict(dweights=A + 4),
    dict(weights=0, ldw=1)])
def test_combine_grad_refuses(bad):
    _refused("sgemm_f32_route_combine_grad", GRAD, bad, GRAD)


GROUPED = dict(transb=0, rows=8, N=16, K=32, experts=3, offsets=A, alpha=1.0, a=B, lda=32, b=C,
               ldb=16, strideb=512, beta=0.0, c=D, ldc=16)


@pytest.mark.parametrize("bad", [
    dict(transb=2), dict(rows=-1), dict(N=-1), dict(K=-1), dict(experts=-1), dict(offsets=0),
    dict(a=0), dict(b=0), dict(c=0), dict(lda=31), dict(ldb=15), dict(ldc=15),
    dict(transb=1, ldb=31), dict(strideb=-1), dict(c=B + 128), dict(c=C + 2 * 512 * 4 + 64),
    dict(c=A + 12)])
def test_grouped_refuses(bad):
    _refused("sgemm_f32_grouped", GROUPED, bad, GROUPED)


GROUPED_TA = dict(rows=8, M=32, N=16, experts=3, offsets=A, alpha=1.0, a=B, lda=32, d=C, ldd=16,
                  beta=0.0, c=D, ldc=16, stridec=512)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(M=-1), dict(N=-1), dict(experts=-1), dict(offsets=0), dict(a=0),
    dict(d=0), dict(c=0), dict(lda=31), dict(ldd=15), dict(ldc=15), dict(stridec=511),
    dict(stridec=-512), dict(c=B + 128), dict(c=C + 64), dict(a=D + 2 * 512 * 4 + 64)])
def test_grouped_ta_refuses(bad):
    _refused("sgemm_f32_grouped_ta", GROUPED_TA, bad, GROUPED_TA)


W4 = dict(M=8, N=16, K=64, a=A, lda=64, packed=B, group=32, scale_type=1, zeros=0, c=C, ldc=16)
W4E = dict(rows=8, N=16, K=64, experts=3, offsets=D, a=A, lda=64, packed=B, group=32, scale_type=1,
           zeros=0, c=C, ldc=16)
BAD_FORMAT = [dict(group=0), dict(group=16), dict(group=96), dict(group=-32), dict(scale_type=3),
              dict(scale_type=-1), dict(N=-1), dict(K=-1)]


@pytest.mark.parametrize("bad", BAD_FORMAT + [
    dict(M=-1), dict(a=0), dict(packed=0), dict(packed=B + 8), dict(c=0), dict(lda=63),
    dict(ldc=15), dict(c=A + 128), dict(c=B + 1024)])
def test_w4_refuses(bad):
    _refused("sgemm_f32_w4", W4, bad, W4)


@pytest.mark.parametrize("bad", BAD_FORMAT + [
    dict(rows=-1), dict(experts=-1), dict(offsets=0), dict(a=0), dict(packed=0), dict(c=0),
    dict(lda=63), dict(ldc=15), dict(c=A + 128), dict(c=D + 8),
    dict(c=B + 2 * 1152 + 64)])  # inside the third matrix
def test_w4_experts_refuses(bad):
    _refused("sgemm_f32_w4_experts", W4E, bad, W4E)


PACK = dict(experts=2, N=16, K=64, group=32, codes=A, scales=B, scale_type=1, zeros=C, packed=D,
            packed_bytes=1 << 20)
QUANTIZE = dict(experts=2, N=16, K=64, group=32, b=A, ldb=16, strideb=1024, scale_type=1, zeros=0,
                packed=D, packed_bytes=1 << 20)
UNPACK = dict(experts=2, N=16, K=64, group=32, scale_type=1, zeros=0, packed=D,
              packed_bytes=1 << 20, b=A, ldb=16, strideb=1024)


@pytest.mark.parametrize("bad", BAD_FORMAT + [
    dict(experts=-1), dict(codes=0), dict(scales=0), dict(packed=0), dict(packed=D + 8),
    dict(scales=B + 1), dict(packed_bytes=2 * (1024 + 4 * 16 * 3) - 1), dict(packed=A + 256),
    dict(codes=D + 16), dict(zeros=D + 16), dict(scales=D + 16)])
def test_pack_refuses(bad):
    _refused("sgemm_f32_w4_pack", PACK, bad, PACK)


@pytest.mark.parametrize("bad", BAD_FORMAT + [
    dict(experts=-1), dict(b=0), dict(ldb=15), dict(strideb=-1), dict(packed=0),
    dict(packed_bytes=2 * (1024 + 4 * 16 * 2) - 1), dict(b=D + 16)])
def test_quantize_refuses(bad):
    _refused("sgemm_f32_w4_quantize", QUANTIZE, bad, QUANTIZE)


@pytest.mark.parametrize("bad", BAD_FORMAT + [
    dict(experts=-1), dict(b=0), dict(ldb=15), dict(strideb=1023), dict(packed=0),
    dict(packed_bytes=2 * (1024 + 4 * 16 * 2) - 1), dict(b=D + 16)])
def test_unpack_refuses(bad):
    _refused("sgemm_f32_w4_unpack", UNPACK, bad, UNPACK)


def test_packed_size():
    # one record of 128 k x 16 columns: 1024 bytes of codes, 16 scales and zero points a part
    size = sg.sgemm_f32_w4_packed_size
    assert size(1, 16, 128, 128, _binding.W4_SCALE_F16, 0) == 1024 + 32
    assert size(1, 16, 128, 128, _binding.W4_SCALE_F32, 1) == 1024 + 64 + 16
    assert size(1, 16, 128, 32, _binding.W4_SCALE_BF16, 1) == 1024 + 4 * (32 + 16)
    assert size(1, 16, 128, 1024, _binding.W4_SCALE_F16, 0) == 1024 + 32
    assert size(3, 17, 129, 64, _binding.W4_SCALE_F16, 0) == 3 * 2 * 2 * (1024 + 2 * 32)
    assert size(0, 16, 128, 128, 0, 0) == 0 and size(1, 0, 128, 128, 0, 0) == 0
    for bad in [(-1, 16, 16, 32, 0, 0), (1, -1, 16, 32, 0, 0), (1, 16, 16, 48, 0, 0),
                (1, 16, 16, 32, 3, 0), (MAX, MAX, MAX, 32, 0, 0)]:
        assert size(*bad) == 0


def test_overlap_found_when_the_extent_passes_64_bits():
    # rows of 2^31 - 1 floats from 2^62 on reach past the top of the address space
    a = 1 << 62
    args = {**GROUPED, "rows": MAX, "lda": MAX, "a": a, "c": a + 4096}
    assert sg.sgemm_f32_grouped(*args.values()) == INVALID


def test_empty_calls_enqueue_nothing():
    zero = {**GATHER, "tokens": 0, "position": 0, "x": 0, "rows": 0}
    assert sg.sgemm_f32_route_gather(*zero.values()) == 0
    zero = {**GATHER, "width": 0, "x": 0, "rows": 0}
    assert sg.sgemm_f32_route_gather(*zero.values()) == 0
    zero = {**COMBINE, "tokens": 0, "position": 0, "rows": 0, "out": 0}
    assert sg.sgemm_f32_route_combine(*zero.values()) == 0
    zero = {**GRAD, "drows": 0, "dweights": 0}
    assert sg.sgemm_f32_route_combine_grad(*zero.values()) == 0
    for nothing in (dict(rows=0), dict(N=0), dict(experts=0)):
        assert sg.sgemm_f32_grouped(*{**GROUPED, **nothing, "a": 0, "b": 0}.values()) == 0
        assert sg.sgemm_f32_w4_experts(*{**W4E, **nothing, "a": 0}.values()) == 0
    for nothing in (dict(M=0), dict(N=0), dict(experts=0)):
        assert sg.sgemm_f32_grouped_ta(*{**GROUPED_TA, **nothing}.values()) == 0
    assert sg.sgemm_f32_w4(*{**W4, "M": 0, "a": 0, "packed": 0, "c": 0}.values()) == 0
    assert sg.sgemm_f32_w4_pack(*{**PACK, "N": 0, "packed": 0}.values()) == 0


def test_no_device_is_an_error_not_a_crash():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for entry, args in [("sgemm_f32_route_gather", GATHER), ("sgemm_f32_route_combine", COMBINE),
                        ("sgemm_f32_route_combine_grad", GRAD), ("sgemm_f32_grouped", GROUPED),
                        ("sgemm_f32_grouped_ta", GROUPED_TA), ("sgemm_f32_w4", W4),
                        ("sgemm_f32_w4_experts", W4E), ("sgemm_f32_w4_pack", PACK),
                        ("sgemm_f32_w4_quantize", QUANTIZE), ("sgemm_f32_w4_unpack", UNPACK)]:
        st = getattr(sg, entry)(*args.values())
        assert st not in (0, INVALID), (entry, st)


def test_torch_layer_refuses_tensors_of_the_host_and_of_other_types():
    torch = pytest.importorskip("torch")
    ids = torch.zeros((4, 2), dtype=torch.int32)
    x = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="GPU"):
        sg.sort_by_expert(ids, 4)
    with pytest.raises(TypeError, match="int32"):
        sg.sort_by_expert(ids.long(), 4)
    r = sg.Routing(torch.zeros(5, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), ids)
    for f in (lambda: sg.gather_rows(x, r), lambda: sg.combine_rows(x, r),
              lambda: sg.grouped_matmul(x, torch.zeros((4, 8, 8)), r.offsets),
              lambda: sg.grouped_matmul_ta(x, x, r.offsets),
              lambda: sg.w4_quantize(torch.zeros((64, 16))),
              lambda: sg.w4_pack(torch.zeros((32, 16), dtype=torch.uint8), torch.zeros((2, 16)),
                                 K=64, group=32)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(TypeError):
        sg.grouped_matmul(x.double(), torch.zeros((4, 8, 8)), r.offsets)


LARGEST = 2**31 - 65537


@pytest.mark.parametrize("entry,base,sizes", [
    ("sgemm_f32_route_sort", SORT, ["tokens", "experts"]),
    ("sgemm_f32_route_gather", GATHER, ["tokens", "width"]),
    ("sgemm_f32_route_combine", COMBINE, ["tokens", "width"]),
    ("sgemm_f32_grouped", GROUPED, ["rows", "N", "K", "experts"]),
    ("sgemm_f32_grouped_ta", GROUPED_TA, ["rows", "M", "N", "experts"]),
    ("sgemm_f32_w4", W4, ["M", "N", "K"]),
    ("sgemm_f32_w4_experts", W4E, ["rows", "N", "K", "experts"])])
def test_sizes_that_do_not_leave_room_for_a_block_are_refused(entry, base, sizes):
    one = {k: 1 for k in base if k in ("tokens", "top", "width", "rows", "M", "N", "K", "experts")}
    row = {"ldids": "top", "ldw": "top", "ldx": "width", "ldrows": "width", "ldout": "width",
           "lda": "M" if "d" in base else "K", "ldb": "N", "ldc": "N", "ldd": "N"}
    for size in sizes:
        for value in (LARGEST + 1, MAX):
            # nothing else is wrong: rows as long as they must be, arrays of 8 GiB at most
            lds = {ld: value if row[ld] == size else 1 for ld in base if ld in row}
            _refused(entry, base, {**one, **lds, size: value}, base)


def test_more_pairs_than_fit_are_refused():
    pairs = {"tokens": 46341, "top": 46341}
    _refused("sgemm_f32_route_sort", SORT, {**pairs, "ldids": 46341}, SORT)
    _refused("sgemm_f32_route_gather", GATHER, pairs, GATHER)
    _refused("sgemm_f32_route_combine", COMBINE, {**pairs, "ldw": 46341}, COMBINE)
    _refused("sgemm_f32_route_combine_grad", GRAD, {**pairs, "ldw": 46341}, GRAD)


def test_packed_size_of_sizes_that_are_refused():
    for experts, N, K in [(LARGEST + 1, 1, 1), (1, LARGEST + 1, 1), (1, 1, LARGEST + 1)]:
        assert sg.sgemm_f32_w4_packed_size(experts, N, K, 128, 0, 0) == 0
    assert sg.sgemm_f32_w4_packed_size(1, 1, LARGEST, 128, 0, 0) > LARGEST // 2


def test_more_blocks_than_a_launch_holds_are_refused():
    far = [(i + 1) << 50 for i in range(5)]
    # 2^24 row blocks of a work-group of 256 work-items each, and twice as many column blocks
    rows = 1 << 29
    assert sg.sgemm_f32_grouped(0, rows, 64, 4, rows // 32, far[0], 1.0, far[1], 4, far[2], 64, 0,
                                0.0, far[3], 64, 0) == INVALID
    assert sg.sgemm_f32_w4_experts(rows, 64, 128, rows // 2, far[0], far[1], 128, far[2], 128, 0, 0,
                                   far[3], 64, 0) == INVALID


def test_a_stream_of_another_gpu_is_refused():
    """A kernel on it would run on that GPU, over memory of this one."""
    torch = pytest.importorskip("torch")
    from dense_fp32_matrix_f32_amd._tensors import launch_stream

    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0x10

    for index in (0, 2):
        with pytest.raises(ValueError, match="stream"):
            launch_stream(Stream(), index)


@pytest.mark.parametrize("experts", [896, 897, 5000, 802815, 802816, 719323135, 719323136,
                                     2**31 - 65537])
def test_digits_of_the_sort_for_many_experts(experts):
    """From 896 experts on the pairs are sorted by digits: the workspace holds the counts of
    a digit for each of the chunks, and the pairs between two digits."""
    tokens, top = 1 << 20, 8
    pairs = tokens * top
    need = sg.sgemm_f32_route_workspace_size(tokens, top, experts)
    base, rest = divmod(need // 4 - pairs, 128)
    assert rest == 0 and 2 <= base <= 896
    digits = next(d for d in range(1, 9) if 896**d > experts)
    assert base**digits > experts and (base - 1)**digits <= experts
    # one chunk, by digits or with a work-group for each expert
    assert sg.sgemm_f32_route_workspace_size(100, 8, experts) == (3200 if experts >= 5000 else 0)
    assert sg.sgemm_f32_route_workspace_size(0, 8, experts) == 0
    if experts < 5000:
        return
    big = {**SORT, "tokens": 100, "top": 8, "ldids": 8, "experts": experts, "ws_bytes": 3200}
    offsets_end = B + 4 * (experts + 1)
    assert offsets_end <= C
    for bad in [dict(ws=0), dict(ws_bytes=3199), dict(ws=E + 4), dict(ws=A + 16), dict(ws=C + 16),
                dict(ws=offsets_end // 16 * 16 - 16)]:
        _refused("sgemm_f32_route_sort", big, bad, SORT)
