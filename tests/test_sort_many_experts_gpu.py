"""Pairs sorted for more experts than one pass takes, against a stable sort by torch."""
import numpy as np
import pytest

import dense_fp32_matrix_f32_amd as sg
from gpu_helpers import log, torch_cuda

pytestmark = pytest.mark.gpu


def check(ids, experts):
    torch = torch_cuda()
    r = sg.sort_by_expert(ids, experts)
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= experts), experts, flat)
    sorted_key, order = torch.sort(key, stable=True)
    kept = int((key < experts).sum())
    order[kept:] = -1
    assert torch.equal(r.order.long(), order)
    position = torch.full_like(flat, -1)
    position[order[:kept]] = torch.arange(kept, device="cuda")
    assert torch.equal(r.position.reshape(-1).long(), position)
    # offsets in pieces, so that 64-bit copies of many of them fit
    for lo in range(0, experts + 1, 1 << 26):
        hi = min(lo + (1 << 26), experts + 1)
        want = torch.searchsorted(sorted_key, torch.arange(lo, hi, device="cuda"))
        assert torch.equal(r.offsets[lo:hi].long(), want)


def ids_of(tokens, top, experts, seed, skew):
    """Uneven experts, some pairs dropped, the last experts among them."""
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand((tokens, top), generator=g, device="cuda", dtype=torch.float64) ** skew
    ids = (u * experts).long().clamp(max=experts - 1)
    ids[torch.rand((tokens, top), generator=g, device="cuda") < 0.05] = experts - 1
    ids = ids.to(torch.int32)
    out = torch.rand((tokens, top), generator=g, device="cuda") < 0.1
    ids[out] = torch.tensor([-1, -2**31, experts, 2**31 - 1], dtype=torch.int32,
                            device="cuda")[torch.randint(0, 4, (int(out.sum()),), generator=g,
                                                         device="cuda")]
    return ids


@pytest.mark.parametrize("experts", [
    895, 896, 897, 1023, 1024, 5000, 65536, 802815, 802816, 3000017])
@pytest.mark.parametrize("tokens,top", [(1, 1), (5, 8), (2048, 3), (2049, 3), (40001, 5)])
def test_sort(tokens, top, experts):
    log(f"[gpu] sort {tokens} x {top}, {experts} experts")
    for skew in (1, 4):
        check(ids_of(tokens, top, experts, tokens + experts, skew), experts)


def test_as_many_pairs_as_experts():
    """A million of each: a pass over all pairs for each expert would not end in useful time."""
    log("[gpu] sort 2^20 x 4, 2^20 experts")
    check(ids_of(1 << 20, 4, 1 << 20, 3, 1), 1 << 20)


@pytest.mark.parametrize("tokens", [3, 3000])
def test_experts_of_four_digits(tokens):
    experts = 719323136 + 11
    log(f"[gpu] sort {tokens} x 3, {experts} experts")
    check(ids_of(tokens, 3, experts, 4, 1), experts)


def test_no_pairs_and_one_expert_for_all():
    torch = torch_cuda()
    empty = sg.sort_by_expert(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 70000)
    assert empty.offsets.eq(0).all() and empty.offsets.numel() == 70001
    for value in (-1, 0, 4999, 5000):
        check(torch.full((7001, 2), value, dtype=torch.int32, device="cuda"), 5000)
    wide = torch.full((5000, 7), 3, dtype=torch.int32, device="cuda")  # a row stride
    wide[:, :2] = ids_of(5000, 2, 2000, 8, 1)
    check(wide[:, :2], 2000)


def test_captured():
    """Two sorts in one graph, replayed on new ids."""
    torch = torch_cuda()
    held = [ids_of(3000, 4, 3000, s, 1) for s in (1, 2)]
    for t in held:
        sg.sort_by_expert(t, 3000)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [sg.sort_by_expert(t, 3000) for t in held]
    for s in range(4):
        for i, t in enumerate(held):
            t.copy_(ids_of(3000, 4, 3000, 10 * s + i, 2))
        for r in out:
            for t in r:
                t.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        for t, r in zip(held, out):
            for a, b in zip(r, sg.sort_by_expert(t, 3000)):
                assert torch.equal(a, b)
