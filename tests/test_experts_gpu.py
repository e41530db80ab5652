"""Rows sorted by expert and back, and the experts' products, against plain
computations in 64 bits on the host.

Tolerances.  A sum of n fp32 products, in any order and with fused or separate
rounding, is within (n + 1) * 2^-24 / (1 - (n + 1) * 2^-24) of the sum of the
products' magnitudes (each product meets at most n roundings); alpha and beta*C
add two more.  `bound()` uses n + 4 and 1.01 for the denominator (n < 2^17)."""
import itertools

import numpy as np
import pytest

import dense_fp32_matrix_f32_amd as sg
from gpu_helpers import log, torch_cuda

pytestmark = pytest.mark.gpu

SENT = float(np.float32(-7.25e30))


def bound(n, magnitude):
    return 1.01 * (n + 4) * 2.0**-24 * magnitude + 1e-37


def close(got, want, n, magnitude, what):
    got = got.double().cpu().numpy() if hasattr(got, "cpu") else got
    off = np.abs(got - want)
    bad = off > bound(n, magnitude)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, the worst by "
                           f"{float((off / np.maximum(bound(n, magnitude), 1e-300)).max()):.3g} "
                           "of the bound")


def plain_sort(ids, experts):
    tokens, top = ids.shape
    flat = ids.reshape(-1)
    order = [f for e in range(experts) for f in np.flatnonzero(flat == e)]
    position = np.full(flat.size, -1, np.int64)
    position[order] = np.arange(len(order))
    offsets = np.array([np.count_nonzero((flat >= 0) & (flat < e)) for e in range(experts + 1)])
    return offsets, np.array(order + [-1] * (flat.size - len(order)), np.int64), \
        position.reshape(tokens, top)


def check_sort(ids, experts, dev_ids=None):
    torch = torch_cuda()
    dev = torch.from_numpy(ids).cuda() if dev_ids is None else dev_ids
    r = sg.sort_by_expert(dev, experts)
    offsets, order, position = plain_sort(ids, experts)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.position.cpu().numpy(), position)
    return r


def make_ids(rng, tokens, top, experts, dropped=0.1, skew=0):
    p = np.exp(-skew * np.arange(experts) / max(1, experts))
    ids = rng.choice(experts, size=(tokens, top), p=p / p.sum()).astype(np.int32)
    out = rng.random((tokens, top)) < dropped
    return np.where(out, rng.choice(np.array([-1, experts, 2**31 - 1, -2**31], np.int64),
                                    size=out.shape), ids).astype(np.int32)


@pytest.mark.parametrize("tokens,top,experts", [
    (1, 1, 1), (1, 8, 64), (3, 2, 5), (63, 1, 2), (64, 1, 3), (65, 4, 64), (127, 8, 65),
    (1000, 3, 17), (1024, 1, 256), (2049, 2, 7), (5000, 8, 300), (20000, 1, 1), (33333, 3, 129),
    (4096, 8, 1000), (70001, 2, 64), (300, 2, 5000),
    (2047, 3, 17), (2049, 3, 895), (30001, 3, 511), (30001, 3, 512), (9999, 7, 895)])
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_sort(tokens, top, experts, dropped):
    log(f"[gpu] sort {tokens} x {top}, {experts} experts, dropped {dropped}")
    rng = np.random.default_rng(tokens * 31 + top)
    check_sort(make_ids(rng, tokens, top, experts, dropped, skew=3), experts)


def test_sort_edge_inputs():
    torch = torch_cuda()
    for tokens, top, experts in [(777, 2, 9), (9000, 4, 70)]:
        check_sort(np.full((tokens, top), 4, np.int32), experts)       # all to one expert
        check_sort(np.full((tokens, top), -1, np.int32), experts)      # all dropped
        check_sort(np.full((tokens, top), 5, np.int32), 0)             # no expert at all
        desc = np.sort(make_ids(np.random.default_rng(1), tokens, top, experts), axis=None)[::-1]
        check_sort(np.ascontiguousarray(desc.reshape(tokens, top)), experts)
        # the same expert twice for a token
        check_sort(np.repeat(make_ids(np.random.default_rng(2), tokens, 1, experts), top, 1),
                   experts)
        # a row stride
        wide = torch.full((tokens, top + 3), 3, dtype=torch.int32, device="cuda")
        ids = make_ids(np.random.default_rng(3), tokens, top, experts)
        wide[:, :top] = torch.from_numpy(ids).cuda()
        check_sort(ids, experts, wide[:, :top])
    empty = sg.sort_by_expert(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 6)
    assert empty.offsets.tolist() == [0] * 7 and empty.order.numel() == 0


def routing_of(tokens, top, experts, seed, dropped=0.15):
    return check_sort(make_ids(np.random.default_rng(seed), tokens, top, experts, dropped), experts)


def padded(torch, x, pad, offset=0, fill=SENT):
    """x as a view of a wider buffer of sentinels, starting `offset` floats into it."""
    r, c = x.shape
    buf = torch.full((r * (c + pad) + offset + 8,), fill, dtype=torch.float32, device="cuda")
    view = buf[offset:offset + r * (c + pad)].view(r, c + pad)[:, :c]
    view.copy_(x)
    return view, buf


WIDTHS = [1, 3, 4, 63, 64, 255, 256, 257, 1000, 1024, 2048, 4099]


@pytest.mark.parametrize("tokens,top,experts", [(1, 1, 2), (1, 8, 16), (7, 2, 3), (130, 3, 8)])
@pytest.mark.parametrize("width", WIDTHS)
def test_rows_there_and_back(tokens, top, experts, width):
    torch = torch_cuda()
    log(f"[gpu] rows {tokens} x {top} of {width}")
    g = torch.Generator().manual_seed(width * 7 + tokens)
    r = routing_of(tokens, top, experts, seed=tokens + width)
    n = tokens * top
    order, position = r.order.cpu().numpy(), r.position.cpu().numpy()
    kept = int(r.offsets[-1])
    for pad, offset in [(0, 0), (5, 0), (4, 4), (1, 3)]:
        x, _ = padded(torch, torch.randn((tokens, width), generator=g), pad, offset)
        y, ybuf = padded(torch, torch.randn((n, width), generator=g), pad, offset)
        w, _ = padded(torch, torch.rand((tokens, top), generator=g), pad)
        dy, _ = padded(torch, torch.randn((tokens, width), generator=g), pad, offset)
        # places of no pair hold values that must reach no result
        y[kept:] = float("nan")
        out, obuf = padded(torch, torch.full((n, width), SENT), pad, offset)
        sg.gather_rows(x, r, out=out)
        want = np.full((n, width), SENT, np.float32)
        want[:kept] = x.cpu().numpy()[order[:kept] // top]
        assert np.array_equal(out.cpu().numpy(), want)
        assert int((obuf != SENT).sum()) == int((torch.from_numpy(want) != SENT).sum())

        Y, W, DY = (t.double().cpu().numpy() for t in (y, w, dy))
        there = (position >= 0)[:, :, None]
        picked = np.where(there, Y[np.maximum(position, 0)], 0.0)
        for weights in (w, None):
            Wm = W if weights is not None else np.ones_like(W)
            back, bbuf = padded(torch, torch.zeros((tokens, width)), pad, offset)
            sg.combine_rows(y, r, weights, out=back)
            terms = picked * Wm[:, :, None]
            close(back, terms.sum(1), top, np.abs(terms).sum(1), "combine")
            back[:] = SENT
            assert int((bbuf != SENT).sum()) == 0, "combine wrote outside its result"

            drows, dbuf = padded(torch, torch.full((n, width), SENT), pad, offset)
            got, dw = sg.combine_rows_grad(dy, y, r, weights, drows=drows)
            want = np.full((n, width), SENT)
            flat = order[:kept]
            want[:kept] = Wm.reshape(-1)[flat][:, None] * DY[flat // top]
            close(got[:kept], want[:kept], 1, np.abs(want[:kept]), "drows")
            got[:kept] = SENT
            assert int((dbuf != SENT).sum()) == 0, "combine_grad wrote outside its result"
            if weights is None:
                assert dw is None
            else:
                terms = picked * DY[:, None, :]
                close(dw, terms.sum(2), width, np.abs(terms).sum(2), "dweights")


def test_combine_of_a_token_without_experts_is_zero():
    torch = torch_cuda()
    ids = torch.tensor([[-1, -1], [0, 1], [9, -5]], dtype=torch.int32, device="cuda")
    r = sg.sort_by_expert(ids, 2)
    y = torch.full((6, 70), float("inf"), device="cuda")
    y[:2] = 2.0
    w = torch.full((3, 2), float("nan"), device="cuda")
    w[1] = 0.5
    out = sg.combine_rows(y, r, w)
    assert out[0].eq(0).all() and out[2].eq(0).all() and out[1].eq(2).all()
    drows, dw = sg.combine_rows_grad(torch.ones((3, 70), device="cuda"), y, r, w)
    assert dw.tolist() == [[0, 0], [140, 140], [0, 0]]


def test_places_outside_the_rows_count_as_dropped():
    """Positions that no sort writes are never followed out of bounds."""
    torch = torch_cuda()
    bad = torch.tensor([[0, 6], [2**31 - 1, -2**31], [3, -1]], dtype=torch.int32, device="cuda")
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    r = sg.Routing(none, none, bad)
    x = torch.arange(3, dtype=torch.float32, device="cuda")[:, None].expand(3, 300).contiguous()
    out = torch.full((6, 300), SENT, device="cuda")
    sg.gather_rows(x, r, out=out)
    assert out[:, 7].tolist() == [0.0, SENT, SENT, 2.0, SENT, SENT]
    y = torch.arange(1, 7, dtype=torch.float32, device="cuda")[:, None].expand(6, 300).contiguous()
    assert sg.combine_rows(y, r)[:, 299].tolist() == [1.0, 0.0, 4.0]
    drows = torch.full((6, 300), SENT, device="cuda")
    _, dw = sg.combine_rows_grad(torch.ones_like(x), y, r, torch.ones((3, 2), device="cuda"),
                                 drows=drows)
    assert drows[:, 0].tolist() == [1.0, SENT, SENT, 1.0, SENT, SENT]
    assert dw.tolist() == [[300, 0], [0, 0], [1200, 0]]


# ---- the experts' products ---------------------------------------------------------------------

GROUPS = {"even": lambda R, E: np.linspace(0, R, E + 1).astype(np.int64),
          "one has all": lambda R, E: np.array([0] * (E // 2 + 1) + [R] * (E - E // 2)),
          "ragged": lambda R, E: np.concatenate([[0], np.sort(np.random.default_rng(R + E).integers(
              0, R + 1, E - 1)), [R]]) if E > 1 else np.array([0, R]),
          "rows of no expert": lambda R, E: np.linspace(R // 5, R - R // 4, E + 1).astype(np.int64)}


def int_matrix(rng, *shape):
    return rng.integers(-4, 5, shape).astype(np.float32)


def plain_grouped(A, B, offsets, C, alpha, beta):
    out = C.copy()
    mag = np.zeros_like(C)
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        out[lo:hi] = alpha * (A[lo:hi] @ B[e]) + (beta * C[lo:hi] if beta else 0)
        mag[lo:hi] = abs(alpha) * (np.abs(A[lo:hi]) @ np.abs(B[e])) + abs(beta) * np.abs(C[lo:hi])
    return out, mag


SHAPES = [(1, 1, 1, 1), (1, 8, 8, 3), (5, 17, 33, 2), (16, 64, 64, 4), (65, 130, 100, 3),
          (200, 96, 257, 5), (333, 257, 63, 70), (130, 4, 500, 4), (64, 1000, 2, 2),
          (700, 200, 72, 8), (48, 520, 1040, 16),
          # few rows of each of many experts
          (300, 257, 70, 200), (700, 1000, 33, 100), (1000, 5, 130, 600), (500, 68, 1, 300),
          (2000, 130, 64, 256)]


@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("rows,N,K,experts", SHAPES)
def test_grouped(rows, N, K, experts, groups):
    torch = torch_cuda()
    rng = np.random.default_rng(rows + N + K)
    offsets = GROUPS[groups](rows, experts)
    dev_off = torch.from_numpy(offsets.astype(np.int32)).cuda()
    for kind, trans, (alpha, beta), pad in itertools.product(
            ("ints", "normal"), (False, True), ((1.0, 0.0), (0.5, -2.0)), (0, 3)):
        if kind == "ints":
            A, B, C = int_matrix(rng, rows, K), int_matrix(rng, experts, K, N), int_matrix(rng, rows, N)
        else:
            A, B, C = (rng.standard_normal(s).astype(np.float32)
                       for s in ((rows, K), (experts, K, N), (rows, N)))
        log(f"[gpu] grouped {rows} x {N} x {K}, {experts} experts, {groups}, {kind} "
            f"{'T' if trans else 'N'} beta {beta} pad {pad}")
        dA, _ = padded(torch, torch.from_numpy(A), pad, offset=pad % 2)
        dC, buf = padded(torch, torch.from_numpy(C), pad, offset=pad)
        if beta == 0.0:
            dC[offsets[0]:offsets[-1]] = float("nan")  # not read
        dB = torch.from_numpy(np.ascontiguousarray(B.transpose(0, 2, 1)) if trans else B).cuda()
        if pad:  # matrices inside wider ones
            wide = torch.full((experts, dB.shape[1] + 1, dB.shape[2] + pad), float("nan"),
                              device="cuda")
            wide[:, :-1, :-pad] = dB
            dB = wide[:, :-1, :-pad]
        if trans:
            dB = dB.transpose(1, 2)
        sg.grouped_matmul(dA, dB, dev_off, out=dC, alpha=alpha, beta=beta)
        want, mag = plain_grouped(A.astype(np.float64), B.astype(np.float64), offsets,
                                  C.astype(np.float64), alpha, beta)
        if kind == "ints":
            assert np.array_equal(dC.double().cpu().numpy(), want)
        else:
            close(dC, want, K, mag, "grouped")
        dC[:] = SENT
        assert int((buf != SENT).sum()) == 0, "wrote outside C"



@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("rows,N,K,experts", [(200, 300, 33, 150), (200, 300, 40, 150), (9, 20, 33, 3)])
def test_grouped_values_that_are_not_finite(rows, N, K, experts, trans):
    """An infinity in the last row of a matrix, or in the first row of the next one, is met only by
    the values of A that belong to it; one in A stays in its row."""
    torch = torch_cuda()
    rng = np.random.default_rng(K)
    offsets = GROUPS["uneven"](rows, experts) if "uneven" in GROUPS else \
        np.sort(np.concatenate([[0], rng.integers(0, rows + 1, experts - 1), [rows]]))
    A, B = int_matrix(rng, rows, K), int_matrix(rng, experts, K, N)
    A[:, K - 1] = 1.0
    B[1::3, K - 1, N // 2] = np.inf
    B[1::3, 0, N - 1] = -np.inf
    A[:, 0] = 2.0
    A[rows // 2, K // 2] = np.nan
    dB = torch.from_numpy(np.ascontiguousarray(B.transpose(0, 2, 1)) if trans else B).cuda()
    got = sg.grouped_matmul(torch.from_numpy(A).cuda(), dB.transpose(1, 2) if trans else dB,
                            torch.from_numpy(offsets.astype(np.int32)).cuda()).cpu().numpy()
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        for i in range(lo, hi):
            want = (A[i][:, None].astype(np.float64) * B[e]).sum(0)
            assert np.array_equal(got[i].astype(np.float64), want, equal_nan=True), (e, i)


@pytest.mark.parametrize("rows,N,K,experts", [(9001, 200, 330, 2), (620, 130, 1030, 4),
                                              (1500, 300, 333, 16), (90, 530, 2050, 2)])
def test_grouped_on_larger_blocks(rows, N, K, experts):
    """Rows an expert at which the larger blocks are taken, k long enough for their
    steady loops."""
    torch = torch_cuda()
    rng = np.random.default_rng(rows)
    offsets = GROUPS["ragged"](rows, experts)
    dev_off = torch.from_numpy(offsets.astype(np.int32)).cuda()
    A, B, D = int_matrix(rng, rows, K), int_matrix(rng, experts, K, N), int_matrix(rng, rows, N)
    dA, dB, dD = (torch.from_numpy(t).cuda() for t in (A, B, D))
    for trans in (False, True):
        mat = dB.transpose(1, 2).contiguous().transpose(1, 2) if trans else dB
        got = sg.grouped_matmul(dA, mat, dev_off).double().cpu().numpy()
        want, _ = plain_grouped(A.astype(np.float64), B.astype(np.float64), offsets,
                                np.zeros((rows, N)), 1.0, 0.0)
        assert np.array_equal(got, want)
    got = sg.grouped_matmul_ta(dA, dD, dev_off).double().cpu().numpy()
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        assert np.array_equal(got[e], A[lo:hi].T.astype(np.float64) @ D[lo:hi])



@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("rows,N,K,experts", [(9001, 530, 330, 2), (4100, 1000, 129, 16),
                                              (4097, 1030, 40, 3)])
def test_grouped_on_blocks_of_two_sizes(rows, N, K, experts, groups):
    """Many rows of each expert: full blocks, and smaller ones for the rows past them."""
    torch = torch_cuda()
    rng = np.random.default_rng(rows + experts)
    offsets = GROUPS[groups](rows, experts)
    dev_off = torch.from_numpy(offsets.astype(np.int32)).cuda()
    A, B, C = int_matrix(rng, rows, K), int_matrix(rng, experts, K, N), int_matrix(rng, rows, N)
    dB = torch.from_numpy(B).cuda()
    for trans, (alpha, beta) in itertools.product((False, True), ((1.0, 0.0), (0.5, -2.0))):
        mat = dB.transpose(1, 2).contiguous().transpose(1, 2) if trans else dB
        dA, _ = padded(torch, torch.from_numpy(A), 3, offset=1)
        dA[:offsets[0]] = float("nan")  # rows of no expert
        dA[offsets[-1]:] = float("nan")
        dC, buf = padded(torch, torch.from_numpy(C), 1, offset=2)
        sg.grouped_matmul(dA, mat, dev_off, out=dC, alpha=alpha, beta=beta)
        want, _ = plain_grouped(A.astype(np.float64), B.astype(np.float64), offsets,
                                C.astype(np.float64), alpha, beta)
        assert np.array_equal(dC.double().cpu().numpy(), want)
        dC[:] = SENT
        assert int((buf != SENT).sum()) == 0, "wrote outside C"


def test_grouped_on_blocks_of_two_sizes_follows_no_offset_out_of_its_rows():
    torch = torch_cuda()
    rng = np.random.default_rng(1)
    rows, N, K, experts = 4200, 1000, 33, 8
    A, B = int_matrix(rng, rows, K), int_matrix(rng, experts, K, N)
    dA, dB = torch.from_numpy(A).cuda(), torch.from_numpy(B).cuda()
    bad = [-2**31, -1, 100, 4000, 2**31 - 1, 7, 7, 7, -3]
    dC, buf = padded(torch, torch.full((rows, N), 1.0), 3, offset=5)
    sg.grouped_matmul(dA, dB, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=dC)
    want = np.ones((rows, N))
    for e, lo, hi in [(1, 0, 100), (2, 100, 4000), (3, 4000, 4200)]:
        want[lo:hi] = A[lo:hi].astype(np.float64) @ B[e]
    assert np.array_equal(dC.double().cpu().numpy(), want)
    # several experts claim all rows: any result, but inside C
    bad = [0, 2**31 - 1] * (experts // 2) + [0]
    sg.grouped_matmul(dA, dB, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=dC)
    dC[:] = SENT
    assert int((buf != SENT).sum()) == 0, "wrote outside C"


def test_rows_so_long_that_offsets_pass_31_bits():
    torch = torch_cuda()
    rng = np.random.default_rng(2)
    ld, rows, K, N, experts = 36_000_003, 6, 40, 70, 2
    offsets = np.array([0, 2, 6])
    dev_off = torch.from_numpy(offsets.astype(np.int32)).cuda()
    A, B, D = int_matrix(rng, rows, K), int_matrix(rng, experts, K, N), int_matrix(rng, rows, N)
    wide = torch.empty((rows, ld), device="cuda")
    dA = wide[:, :K]
    dA.copy_(torch.from_numpy(A))
    dB = torch.from_numpy(B).cuda()
    want, _ = plain_grouped(A.astype(np.float64), B.astype(np.float64), offsets,
                            np.zeros((rows, N)), 1.0, 0.0)
    for mat in (dB, dB.transpose(1, 2).contiguous().transpose(1, 2)):
        out = torch.empty((rows, ld), device="cuda")[:, 5:5 + N]
        sg.grouped_matmul(dA, mat, dev_off, out=out)
        assert np.array_equal(out.double().cpu().numpy(), want)
        del out
    got = sg.grouped_matmul_ta(dA, torch.from_numpy(D).cuda(), dev_off).double().cpu().numpy()
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        assert np.array_equal(got[e], A[lo:hi].T.astype(np.float64) @ D[lo:hi])


@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("rows,N,M,experts", SHAPES)
def test_grouped_ta(rows, N, M, experts, groups):
    torch = torch_cuda()
    rng = np.random.default_rng(rows * 3 + N + M)
    offsets = GROUPS[groups](rows, experts)
    dev_off = torch.from_numpy(offsets.astype(np.int32)).cuda()
    for kind, (alpha, beta), pad in itertools.product(("ints", "normal"), ((1.0, 0.0), (0.5, -2.0)),
                                                      (0, 3)):
        make = (lambda *s: int_matrix(rng, *s)) if kind == "ints" else \
            (lambda *s: rng.standard_normal(s).astype(np.float32))
        A, D, C = make(rows, M), make(rows, N), make(experts, M, N)
        log(f"[gpu] grouped_ta {rows}: {M} x {N}, {experts} experts, {groups}, {kind} beta {beta} "
            f"pad {pad}")
        dA, _ = padded(torch, torch.from_numpy(A), pad, offset=pad % 2)
        dD, _ = padded(torch, torch.from_numpy(D), pad, offset=pad)
        wide = torch.full((experts, M + 1, N + pad), SENT, device="cuda")
        dC = wide[:, :M, :N]
        dC.copy_(torch.from_numpy(C)) if beta else dC.fill_(float("nan"))
        sg.grouped_matmul_ta(dA, dD, dev_off, out=dC, alpha=alpha, beta=beta)
        want, mag = np.zeros((experts, M, N)), np.zeros((experts, M, N))
        for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            a, d = A[lo:hi].astype(np.float64), D[lo:hi].astype(np.float64)
            want[e] = alpha * (a.T @ d) + beta * C[e]
            mag[e] = abs(alpha) * (np.abs(a).T @ np.abs(d)) + abs(beta) * np.abs(C[e])
        if kind == "ints":
            assert np.array_equal(dC.double().cpu().numpy(), want)
        else:
            close(dC, want, rows, mag, "grouped_ta")
        dC.fill_(SENT)
        assert int((wide != SENT).sum()) == 0, "wrote outside C"


def test_grouped_without_k_or_alpha():
    torch = torch_cuda()
    off = torch.tensor([1, 3, 3, 6], dtype=torch.int32, device="cuda")
    C = torch.full((7, 40), 3.0, device="cuda")
    sg.grouped_matmul(torch.empty((7, 0), device="cuda"), torch.empty((3, 0, 40), device="cuda"),
                      off, out=C)
    assert C[:, 0].tolist() == [3, 0, 0, 0, 0, 0, 3]
    C.fill_(3.0)
    nan = torch.full((7, 5), float("nan"), device="cuda")
    B = torch.full((3, 5, 40), float("nan"), device="cuda")
    sg.grouped_matmul(nan, B, off, out=C, alpha=0.0, beta=2.0)
    assert C[:, 39].tolist() == [3, 6, 6, 6, 6, 6, 3]
    out = torch.full((3, 5, 5), 3.0, device="cuda")
    sg.grouped_matmul_ta(nan, nan, off, out=out, alpha=0.0, beta=2.0)
    assert out.eq(6.0).all()
    none = torch.empty((0, 5), device="cuda")
    zero = sg.grouped_matmul_ta(none, none, torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert zero.shape == (3, 5, 5) and zero.eq(0).all()


def test_grouped_follows_no_offset_out_of_its_rows():
    """Offsets that are no running sum are clamped to the rows there are."""
    torch = torch_cuda()
    rows, K, N = 100, 72, 68
    A = torch.ones((rows, K), device="cuda")
    B = torch.ones((3, K, N), device="cuda")
    for bad, own in [([0, 1000, 2**31 - 1, -5], range(0, 100)), ([-2**31, -1, 50, 70], range(0, 70)),
                     ([90, 20, 10, 400], range(10, 100))]:
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        buf = torch.full((rows + 200, N), SENT, device="cuda")
        sg.grouped_matmul(A, B, off, out=buf[100:200])
        assert int((buf[:100] != SENT).sum()) == 0 and int((buf[200:] != SENT).sum()) == 0
        got = [i for i in range(rows) if float(buf[100 + i, 0]) != SENT]
        assert got == list(own) and buf[100 + own[0], 5] == K
        sg.grouped_matmul_ta(A, A, off)


def test_offsets_that_name_more_rows_than_there_are():
    """Every other expert claims all rows: more blocks than the launch holds.  Nothing
    outside the rows is touched, and rows that are written hold some expert's product."""
    torch = torch_cuda()
    rows, K, N, experts = 200, 40, 300, 150
    off = torch.tensor([0, 2**31 - 1] * (experts // 2) + [0], dtype=torch.int32, device="cuda")
    A, B = torch.ones((rows, K), device="cuda"), torch.ones((experts, K, N), device="cuda")
    buf = torch.full((rows + 400, N), SENT, device="cuda")
    sg.grouped_matmul(A, B, off, out=buf[200:400])
    assert int((buf[:200] != SENT).sum()) == 0 and int((buf[400:] != SENT).sum()) == 0
    inside = buf[200:400]
    assert ((inside == SENT) | (inside == K)).all()
    C = sg.grouped_matmul_ta(A, torch.ones((rows, 24), device="cuda"), off)
    assert C[0::2].eq(rows).all() and C[1::2].eq(0).all()
    w = sg.w4_quantize(torch.full((experts, 64, N), 7.0, device="cuda"), group=32)
    buf.fill_(SENT)
    sg.matmul_w4(torch.ones((rows, 64), device="cuda"), w, offsets=off, out=buf[200:400])
    assert int((buf[:200] != SENT).sum()) == 0 and int((buf[400:] != SENT).sum()) == 0
    inside = buf[200:400]
    assert ((inside == SENT) | (inside == 448)).all()


def test_combine_grad_of_one_side_only():
    """drows or dweights may be left out, and rows with the latter."""
    torch = torch_cuda()
    for tokens, top, width in [(5, 3, 70), (600, 6, 1500), (3, 9, 5000)]:
        r = routing_of(tokens, top, 7, seed=width)
        n = tokens * top
        y, dy = torch.randn((n, width), device="cuda"), torch.randn((tokens, width), device="cuda")
        w = torch.rand((tokens, top), device="cuda")
        drows, dw = torch.full((n, width), SENT, device="cuda"), None
        _, dw = sg.combine_rows_grad(dy, y, r, w, drows=drows)
        one = torch.full((n, width), SENT, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        args = (tokens, top, width, r.position.data_ptr(), w.data_ptr(), top)
        assert sg.sgemm_f32_route_combine_grad(*args, 0, width, dy.data_ptr(), width,
                                               one.data_ptr(), width, 0, s) == 0
        assert torch.equal(one, drows)
        two = torch.empty((tokens, top), device="cuda")
        assert sg.sgemm_f32_route_combine_grad(*args, y.data_ptr(), width, dy.data_ptr(), width, 0,
                                               width, two.data_ptr(), s) == 0
        assert torch.equal(two, dw)
        # no columns: the sums are empty
        two.fill_(SENT)
        assert sg.sgemm_f32_route_combine_grad(tokens, top, 0, r.position.data_ptr(), 0, top, 0, 1,
                                               0, 1, 0, 1, two.data_ptr(), s) == 0
        assert two.eq(0).all()


def test_arrays_beyond_32_bits():
    """Rows past the 2^31st element, and matrices past the 2^32nd byte."""
    torch = torch_cuda()
    tokens, top, width, experts = 270_000, 2, 4096, 3
    ids = torch.randint(0, experts, (tokens, top), dtype=torch.int32, device="cuda")
    r = sg.sort_by_expert(ids, experts)
    x = torch.randint(-8, 9, (tokens, 1), device="cuda").float() + \
        torch.arange(width, device="cuda") % 16
    rows = sg.gather_rows(x, r)
    assert rows.numel() > 2**31
    for t in (0, tokens // 2, tokens - 1):
        for j in range(top):
            assert torch.equal(rows[int(r.position[t, j])], x[t])
    assert torch.equal(rows[-1], x[int(r.order[-1]) // top])
    back = sg.combine_rows(rows, r)
    assert torch.equal(back, 2 * x)
    del back
    w = torch.full((tokens, top), 0.5, device="cuda")
    drows, dw = sg.combine_rows_grad(x, rows, r, w)
    assert torch.equal(drows[-1], 0.5 * x[int(r.order[-1]) // top])
    assert torch.equal(dw[-1].double(), (x[-1].double() ** 2).sum().expand(2))
    del rows, drows, x

    experts, K, N, n = 18, 8192, 8192, 40
    B = torch.zeros((experts, K, N), device="cuda")
    last = torch.randint(-2, 3, (K, N), device="cuda").float()
    B[-1] = last
    A = torch.randint(-2, 3, (n, K), device="cuda").float()
    off = torch.tensor([0] * experts + [n], dtype=torch.int32, device="cuda")
    off[-2] = 3
    for mat in (B, B.transpose(1, 2)):
        C = sg.grouped_matmul(A, mat, off)
        want = A.double() @ (last if mat is B else last.t()).double()
        want[:3] = 0
        assert torch.equal(C.double(), want)
    dB = sg.grouped_matmul_ta(A, C, off)
    assert torch.equal(dB[-1].double(), A[3:].double().t() @ C[3:].double())
    assert dB[-2].eq(0).all() and dB[0].eq(0).all()



def test_more_tokens_than_a_launch_has_places_for():
    """Narrow rows of so many tokens that work-groups take several in turn."""
    torch = torch_cuda()
    tokens, experts = (1 << 25) + (1 << 24) + 5, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(-1, experts, (tokens, 1), dtype=torch.int32, device="cuda", generator=g)
    r = sg.sort_by_expert(ids, experts)
    kept = ids[:, 0] >= 0
    counts = torch.bincount(ids[kept, 0], minlength=experts)
    assert torch.equal(r.offsets[1:].long(), counts.cumsum(0))
    x = torch.randint(-8, 9, (tokens, 1), device="cuda", generator=g).float()
    rows = sg.gather_rows(x, r)
    n = int(r.offsets[-1])
    assert torch.equal(rows[:n, 0], x[r.order[:n].long(), 0])
    w = torch.randint(-3, 4, (tokens, 1), device="cuda", generator=g).float()
    assert torch.equal(sg.combine_rows(rows, r, w)[:, 0], torch.where(kept, w[:, 0] * x[:, 0], 0))
    dout = torch.randint(-8, 9, (tokens, 1), device="cuda", generator=g).float()
    drows, dw = sg.combine_rows_grad(dout, rows, r, w)
    assert torch.equal(drows[:n, 0], (w * dout)[r.order[:n].long(), 0])
    assert torch.equal(dw[:, 0], torch.where(kept, dout[:, 0] * x[:, 0], 0))


def test_sort_for_millions_of_experts():
    torch = torch_cuda()
    experts = (1 << 22) + 17
    ids = torch.tensor([[experts - 1, 3], [1 << 21, experts], [3, 0], [-1, (1 << 21) + 1]],
                       dtype=torch.int32, device="cuda")
    r = sg.sort_by_expert(ids, experts)
    flat = ids.flatten().tolist()
    order = sorted((f for f in range(8) if 0 <= flat[f] < experts), key=lambda f: (flat[f], f))
    assert r.order.tolist() == order + [-1] * (8 - len(order))
    assert r.position.flatten().tolist() == [order.index(f) if f in order else -1 for f in range(8)]
    own = torch.tensor(sorted(flat[f] for f in order), device="cuda")
    want = torch.searchsorted(own, torch.arange(experts + 1, device="cuda"))
    assert torch.equal(r.offsets.long(), want)


def test_one_matrix_for_all_experts():
    torch = torch_cuda()
    rng = np.random.default_rng(5)
    A, B = int_matrix(rng, 90, 40), int_matrix(rng, 40, 70)
    off = torch.tensor([0, 30, 31, 90], dtype=torch.int32, device="cuda")
    C = sg.grouped_matmul(torch.from_numpy(A).cuda(), torch.from_numpy(B).cuda()[None].expand(3, 40, 70), off)
    assert np.array_equal(C.cpu().numpy(), A @ B)


# ---- together ---------------------------------------------------------------------------------


def layer(x, ids, weights, B1, B2, dout=None):
    """A layer of experts: rows out, two products with a ReLU between, rows back; with
    dout, the gradients of x, weights, B1 and B2 too."""
    torch = torch_cuda()
    r = sg.sort_by_expert(ids, B1.shape[0])
    kept = (torch.arange(ids.numel(), device="cuda") < r.offsets[-1])[:, None]
    rows = torch.zeros((ids.numel(), x.shape[1]), device="cuda")
    sg.gather_rows(x, r, out=rows)
    pre = torch.zeros((ids.numel(), B1.shape[2]), device="cuda")
    sg.grouped_matmul(rows, B1, r.offsets, out=pre)
    h = pre.clamp(min=0.0)
    y = torch.zeros((ids.numel(), B2.shape[2]), device="cuda")
    sg.grouped_matmul(h, B2, r.offsets, out=y)
    out = sg.combine_rows(y, r, weights)
    if dout is None:
        return out
    dy = torch.zeros_like(y)
    _, dw = sg.combine_rows_grad(dout, y, r, weights, drows=dy)
    dB2 = sg.grouped_matmul_ta(h, dy, r.offsets)
    dh = torch.zeros_like(h)
    sg.grouped_matmul(dy, B2.transpose(1, 2), r.offsets, out=dh)
    dpre = torch.where((pre > 0) & kept, dh, 0.0)
    dB1 = sg.grouped_matmul_ta(rows, dpre, r.offsets)
    drows = torch.zeros_like(rows)
    sg.grouped_matmul(dpre, B1.transpose(1, 2), r.offsets, out=drows)
    return out, sg.combine_rows(drows, r), dw, dB1, dB2


def plain_layer(x, ids, weights, B1, B2):
    """The same in 64 bits with torch's autograd on the host."""
    torch = torch_cuda()
    out = []
    for t in range(x.shape[0]):
        row = torch.zeros(B2.shape[2], dtype=torch.float64)
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if 0 <= e < B1.shape[0]:
                row = row + weights[t, j] * (torch.relu(x[t] @ B1[e]) @ B2[e])
        out.append(row)
    return torch.stack(out)


def layer_case(tokens, top, experts, width, hidden, seed):
    torch = torch_cuda()
    g = torch.Generator().manual_seed(seed)
    ids = torch.from_numpy(make_ids(np.random.default_rng(seed), tokens, top, experts, 0.1))
    x = torch.randn((tokens, width), generator=g)
    w = torch.rand((tokens, top), generator=g)
    B1 = torch.randn((experts, width, hidden), generator=g) / width**0.5
    B2 = torch.randn((experts, hidden, width), generator=g) / hidden**0.5
    return ids, x, w, B1, B2, torch.randn((tokens, width), generator=g)


@pytest.mark.parametrize("tokens,top,experts,width,hidden", [
    (1, 2, 4, 64, 128), (37, 2, 6, 48, 80), (150, 4, 8, 100, 36)])
def test_layer_of_experts_and_its_gradients(tokens, top, experts, width, hidden):
    torch = torch_cuda()
    ids, x, w, B1, B2, dout = layer_case(tokens, top, experts, width, hidden, 11)
    got = layer(x.cuda(), ids.cuda(), w.cuda(), B1.cuda(), B2.cuda(), dout.cuda())
    leaves = [t.double().requires_grad_() for t in (x, w, B1, B2)]
    out = plain_layer(leaves[0], ids, leaves[1], leaves[2], leaves[3])
    (out * dout.double()).sum().backward()
    want = [out.detach()] + [t.grad for t in leaves]
    # The values pass at most four products of lengths width, hidden, top and width (or
    # the number of rows), each off by (n + 4) 2^-24 of the sum of magnitudes, which is
    # at most sqrt(n) times the values' root mean square: with n <= 600 and values of
    # order one, below 4 * 604 * 2^-24 * sqrt(600) = 3.5e-3 of the largest value.  A ReLU
    # whose argument rounds across zero changes a term of that same size.
    for a, b, name in zip(got, want, ("out", "dx", "dweights", "dB1", "dB2")):
        off = float((a.double().cpu() - b).abs().max())
        assert off <= 3.5e-3 * float(b.abs().max()), (name, off)


def test_layer_gradient_against_differences():
    """The layer is linear in `weights` and in B2: a step of a power of two along small
    integers changes the loss by exactly the gradient's share of it."""
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    ids = torch.from_numpy(make_ids(rng, 20, 2, 4, 0.1)).cuda()
    ints = lambda *s: torch.from_numpy(rng.integers(-2, 3, s).astype(np.float32)).cuda()  # noqa: E731
    x, w, B1, B2, dout = ints(20, 8), ints(20, 2), ints(4, 8, 6), ints(4, 6, 8), ints(20, 8)
    out, dx, dw, dB1, dB2 = layer(x, ids, w, B1, B2, dout)
    step_w, step_B2 = ints(20, 2), ints(4, 6, 8)
    loss = lambda **k: float((layer(x, ids, k.get("w", w), B1, k.get("B2", B2)).double()  # noqa: E731
                              * dout.double()).sum())
    assert loss(w=w + step_w) - loss() == float((dw * step_w).double().sum())
    assert loss(B2=B2 + step_B2) - loss() == float((dB2 * step_B2).double().sum())
    # where no argument of the ReLU is near zero it is linear in x and B1 as well
    x2, B12 = x.abs() + 1, B1.abs() + 1
    _, dx, _, dB1, _ = layer(x2, ids, w, B12, B2, dout)
    loss = lambda a, b: float((layer(a, ids, w, b, B2).double() * dout.double()).sum())  # noqa: E731
    sx, sB1 = ints(20, 8).abs(), ints(4, 8, 6).abs()
    assert loss(x2 + sx, B12) - loss(x2, B12) == float((dx * sx).double().sum())
    assert loss(x2, B12 + sB1) - loss(x2, B12) == float((dB1 * sB1).double().sum())


def test_layer_captured_into_a_graph():
    """The whole layer with its gradients in one HIP graph, replayed on new inputs with
    eager work between the replays."""
    torch = torch_cuda()
    cases = [layer_case(70, 2, 5, 64, 96, seed) for seed in range(4)]
    held = [t.cuda() for t in cases[0]]
    ids, x, w, B1, B2, dout = held
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, ids, w, B1, B2, dout)  # warm up
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer(x, ids, w, B1, B2, dout)
    for case in cases[1:] + cases[:1]:
        for t, new in zip(held, case):
            t.copy_(new)
        want = [t.clone() for t in layer(x, ids, w, B1, B2, dout)]
        torch.cuda.synchronize()
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_calls_on_another_stream():
    torch = torch_cuda()
    s = torch.cuda.Stream()
    x = torch.randn((500, 256), device="cuda")
    ids = torch.from_numpy(make_ids(np.random.default_rng(8), 500, 2, 8, 0.0)).cuda()
    B = torch.randn((8, 256, 128), device="cuda")
    r = sg.sort_by_expert(ids, 8)
    want = sg.combine_rows(sg.grouped_matmul(sg.gather_rows(x, r), B, r.offsets), r)
    torch.cuda.synchronize()
    for _ in range(3):
        r2 = sg.sort_by_expert(ids, 8, stream=s)
        c = sg.grouped_matmul(sg.gather_rows(x, r2, stream=s), B, r2.offsets, stream=s)
        got = sg.combine_rows(c, r2, stream=s)
        del c, r2
        junk = torch.full((1000, 256), float("nan"), device="cuda")
        s.synchronize()
        assert torch.equal(got, want)
        del junk


def test_refusals_of_the_torch_layer():
    torch = torch_cuda()
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    r = sg.sort_by_expert(ids, 3)
    x = torch.zeros((4, 8), device="cuda")
    y = torch.zeros((8, 8), device="cuda")
    B = torch.zeros((3, 8, 8), device="cuda")
    for f in (lambda: sg.gather_rows(y, r), lambda: sg.combine_rows(x, r),
              lambda: sg.gather_rows(x.t(), r), lambda: sg.combine_rows(y, r, weights=x),
              lambda: sg.gather_rows(x, r, out=x), lambda: sg.grouped_matmul(y, B, r.offsets[:2]),
              lambda: sg.grouped_matmul(y[:, :4], B, r.offsets),
              lambda: sg.grouped_matmul(y, B[:, ::2], r.offsets, out=y),
              lambda: sg.grouped_matmul(y, B, r.offsets, beta=1.0),
              lambda: sg.grouped_matmul_ta(y, x, r.offsets),
              lambda: sg.gather_rows(x[:1].expand(4, 8), r),
              lambda: sg.gather_rows(x, sg.Routing(r.offsets, r.order, r.position.t())),
              lambda: sg.combine_rows_grad(x, x, r)):
        with pytest.raises((ValueError, TypeError)):
            f()
    with pytest.raises(sg.SgemmError):
        sg.gather_rows(y[:4], r, out=y)   # overlapping memory
