"""Combination and its gradients where the rows are large enough (256 MB) to be stored past
the caches: odd widths, row strides, bases off 16 bytes, more than four choices, dropped
pairs.  Against 64-bit computations on the GPU.

Tolerance: a sum of n products is within 1.01 * (n + 4) * 2^-24 of the sum of their
magnitudes; one product is rounded once."""
import numpy as np
import pytest

import dense_fp32_matrix_f32_amd as sg
from gpu_helpers import log, torch_cuda

pytestmark = pytest.mark.gpu

SENT = float(np.float32(-7.25e30))


def buffer(rows, cols, pad, offset, fill=SENT):
    torch = torch_cuda()
    buf = torch.full((rows * (cols + pad) + offset + 8,), fill, device="cuda")
    return buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def filled(rows, cols, pad, offset, g):
    torch = torch_cuda()
    view, _ = buffer(rows, cols, pad, offset)
    view.copy_(torch.randn((rows, cols), generator=g, device="cuda"))
    return view


def within(got, want, limit):
    torch = torch_cuda()
    assert torch.isfinite(got).all()
    off = (got.double() - want).abs()
    assert (off <= limit).all(), float((off / limit.clamp(min=1e-300)).max())


def outside_untouched(buf, view):
    view.fill_(SENT)
    assert int((buf != SENT).sum()) == 0, "wrote outside its result"


@pytest.mark.parametrize("tokens,top,width,pad,offset", [
    (30011, 5, 449, 3, 1),     # every row off 16 bytes, a last column past the vectors
    (3001, 9, 2500, 4, 0),     # three rounds of choices, whole vectors
    (16411, 1, 4099, 0, 3),    # one choice, dense odd rows on an odd base
    (150007, 7, 65, 2, 2),     # narrow rows
    (263, 4, 64011, 1, 1)])    # few tokens, wide rows
def test_large_rows(tokens, top, width, pad, offset):
    torch = torch_cuda()
    n = tokens * top
    assert n * width * 4 >= 256 << 20
    log(f"[gpu] {tokens} x {top} rows of {width} past the caches")
    g = torch.Generator(device="cuda").manual_seed(width)
    ids = torch.randint(-2, 12, (tokens, top), generator=g, device="cuda", dtype=torch.int32)
    ids[5] = -1  # a token whose pairs are all dropped
    r = sg.sort_by_expert(ids, 10)
    kept = int(r.offsets[-1])
    assert 0 < kept < n
    there = r.position >= 0
    order = r.order[:kept].long()
    rows = filled(n, width, pad, offset, g)
    rows[kept:] = float("nan")  # rows of no pair reach no result
    w, dout = filled(tokens, top, pad, 0, g), filled(tokens, width, pad, offset, g)
    for weights in (w, None):
        out, obuf = buffer(tokens, width, pad, offset)
        drows, dbuf = buffer(n, width, pad, offset)
        sg.combine_rows(rows, r, weights, out=out)
        _, dw = sg.combine_rows_grad(dout, rows, r, weights, drows=drows)
        assert drows[kept:].eq(SENT).all()
        # in columns, so that the 64-bit copies fit
        want_dw, mag_dw = (torch.zeros((tokens, top), dtype=torch.float64, device="cuda")
                           for _ in range(2))
        for lo in range(0, width, 8192):
            c = slice(lo, min(lo + 8192, width))
            want, mag = (torch.zeros((tokens, c.stop - lo), dtype=torch.float64, device="cuda")
                         for _ in range(2))
            for j in range(top):
                y = rows[:, c][r.position[:, j].clamp(min=0).long()].double()
                y[~there[:, j]] = 0.0
                term = y if weights is None else y * weights[:, j, None].double()
                want += term
                mag += term.abs()
                term = y * dout[:, c].double()
                want_dw[:, j] += term.sum(1)
                mag_dw[:, j] += term.abs().sum(1)
            within(out[:, c], want, 1.01 * (top + 4) * 2.0**-24 * mag)
            one = dout[:, c][order // top]
            exact = one.double() if weights is None else \
                one.double() * weights.reshape(-1)[order][:, None].double()
            within(drows[:kept, c], exact, 2.0**-24 * exact.abs())
        if weights is None:
            assert dw is None
        else:
            within(dw, want_dw, 1.01 * (width + 4) * 2.0**-24 * mag_dw)
            assert dw[~there].eq(0).all()
        assert out[5].eq(0).all()
        outside_untouched(obuf, out)
        outside_untouched(dbuf, drows)
