"""The measured cases of the operators around the matrix product: products with 4-bit weights
(one matrix, or one for each expert), rows sorted by expert and brought back, and the products
of experts.  ``run`` computes them from elementary torch operations in 32 bits, or, where
``own`` is true, through this package's entry points."""
import math

import torch

own = False

SCALES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # 4-bit weights, one matrix
        # one token of a decoder through a square projection: the call whose latency counts
        dict(name="w4 one token", op="w4", rows=1, n=4096, k=4096, group=128, zeros=False, scale="f16"),
        # a few drafted tokens, every size odd, the last group of k cut short
        dict(name="w4 odd sizes", op="w4", rows=5, n=1023, k=4097, group=32, zeros=True, scale="f32"),
        # a batch of sequences that decode together, through a wide matrix
        dict(name="w4 batch", op="w4", rows=16, n=8192, k=8192, group=64, zeros=True, scale="bf16"),
        # a prompt's chunk: enough rows for the arithmetic to count
        dict(name="w4 prompt", op="w4", rows=512, n=8192, k=4096, group=128, zeros=False, scale="f16"),
        # 4-bit weights, one matrix for each expert
        # one token through its eight experts of 64
        dict(name="w4 experts one token", op="w4_experts", tokens=1, top=8, experts=64, n=2048, k=2048, group=128,
             zeros=False, scale="f16"),
        # a decoding batch, its rows spread unevenly
        dict(name="w4 experts batch", op="w4_experts", tokens=64, top=4, experts=16, n=1408, k=4096, group=32,
             zeros=True, scale="f16"),
        # order of the rows
        # a decoding batch of one token: pure latency
        dict(name="sort one token", op="sort", tokens=1, top=8, experts=64, dropped=0.0),
        # a training step's tokens with padding among them, whose rows no expert gets
        dict(name="sort step", op="sort", tokens=32768, top=8, experts=256, dropped=0.1),
        # rows to their experts and back
        # a small serving batch of an odd number of tokens
        dict(name="rows serving", op="rows", tokens=33, top=2, experts=8, width=4096, train=False),
        # a training step: both ways, and both gradients
        dict(name="rows step", op="rows", tokens=8192, top=4, experts=64, width=2048, train=True),
        # the experts' products
        # a serving batch: bound by reading the weights of the experts that have rows
        dict(name="experts serving", op="experts", tokens=24, top=2, experts=8, n=4096, k=2048, train=False),
        # a training step: the product and both gradients, experts of very different sizes
        dict(name="experts step", op="experts", tokens=4096, top=2, experts=8, n=4096, k=2048, train=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the ranges that the listed ones stand for."""
    op = rng.choice(["w4", "w4", "w4_experts", "sort", "rows", "experts"])
    if op in ("w4", "w4_experts"):
        c = dict(op=op, n=_log(rng, 64, 8192), k=_log(rng, 64, 8192), group=rng.choice([32, 64, 128, 256]),
                 zeros=rng.random() < 0.5, scale=rng.choice(["f32", "f16", "bf16"]))
        if op == "w4":
            return dict(c, rows=_log(rng, 1, 512))
        c["experts"] = _log(rng, 2, 64)
        while c["experts"] * c["n"] * c["k"] > 64 * 2048 * 2048:
            c["experts"] = max(2, c["experts"] // 2)
            c["n"] = max(64, c["n"] * 2 // 3)
        return dict(c, tokens=_log(rng, 1, 128), top=rng.randint(1, min(8, c["experts"])))
    experts = _log(rng, 2, 256 if op == "sort" else 64)
    top = rng.randint(1, min(8, experts))
    if op == "sort":
        return dict(op=op, tokens=_log(rng, 1, 32768), top=top, experts=experts, dropped=rng.choice([0.0, 0.02, 0.3]))
    if op == "rows":
        c = dict(op=op, tokens=_log(rng, 1, 8192), top=top, experts=experts, width=_log(rng, 64, 4096),
                 train=rng.random() < 0.5)
        while c["tokens"] * c["top"] * c["width"] > 8192 * 4 * 2048:
            c["tokens"] = c["tokens"] // 2 + 1
        return c
    c = dict(op=op, tokens=_log(rng, 1, 4096), top=top, experts=experts, n=_log(rng, 64, 4096), k=_log(rng, 64, 4096),
             train=rng.random() < 0.5)
    while c["experts"] * c["n"] * c["k"] > 8 * 4096 * 2048:
        c["n"], c["k"] = c["n"] * 2 // 3, c["k"] * 2 // 3
    while c["tokens"] * c["top"] * c["n"] * c["k"] > 4096 * 2 * 4096 * 2048:
        c["tokens"] = c["tokens"] // 2 + 1
    return c


# ---- inputs ---------------------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _router(g, tokens, top, experts):
    """Each token's experts and their weights, as a router with uneven experts gives them."""
    logits = _normal(g, tokens, experts) + 0.5 * _normal(g, experts)
    best, ids = torch.topk(logits, top, dim=1)
    return ids.to(torch.int32).contiguous(), torch.softmax(best, dim=1).contiguous()


def _by_expert(ids, experts):
    """Where each expert's rows begin, the rows' order, and each row's place."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    offsets = torch.zeros(experts + 1, dtype=torch.long, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=experts), 0)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device="cuda")
    return offsets.to(torch.int32), order.to(torch.int32), position.to(torch.int32).reshape(ids.shape)


def _codes(g, experts, k, n):
    """4-bit codes, two rows of k in a byte, spread as a quantised normal weight's are."""
    made = []
    for _ in range(experts):
        q = (8.0 + 2.7 * _normal(g, k + k % 2, n)).round_().clamp_(0, 15).to(torch.uint8)
        made.append(q[0::2] | (q[1::2] << 4))
    return torch.stack(made)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=dict(case))
    op = case["op"]
    if op in ("w4", "w4_experts"):
        n, k, group = case["n"], case["k"], case["group"]
        experts = case.get("experts", 1)
        groups = -(-k // group)
        s["codes"] = _codes(g, experts, k, n)
        s["scales"] = (0.005 + 0.01 * torch.rand((experts, groups, n), generator=g, device="cuda")).to(SCALES[case["scale"]])
        s["zeros"] = torch.randint(6, 11, (experts, groups, n), generator=g, device="cuda", dtype=torch.uint8) \
            if case["zeros"] else None
        rows = case["rows"] if op == "w4" else case["tokens"] * case["top"]
        s["a"] = _normal(g, rows, k)
        if op == "w4_experts":
            ids, _ = _router(g, case["tokens"], case["top"], experts)
            s["offsets"], _, _ = _by_expert(ids, experts)
            s["most"] = int(torch.diff(s["offsets"]).max())
        else:
            s["codes"], s["scales"] = s["codes"][0], s["scales"][0]
            s["zeros"] = s["zeros"][0] if case["zeros"] else None
        if own:
            import dense_fp32_matrix_f32_amd as sg
            s["w"] = sg.w4_pack(s["codes"], s["scales"], s["zeros"], K=k, group=group)
    elif op == "sort":
        ids, _ = _router(g, case["tokens"], case["top"], case["experts"])
        padding = torch.rand(case["tokens"], generator=g, device="cuda") < case["dropped"]
        s["ids"] = torch.where(padding[:, None], -1, ids).contiguous()
    elif op == "rows":
        ids, s["weights"] = _router(g, case["tokens"], case["top"], case["experts"])
        s["offsets"], s["order"], s["position"] = _by_expert(ids, case["experts"])
        rows = case["tokens"] * case["top"]
        s["x"], s["y"] = _normal(g, case["tokens"], case["width"]), _normal(g, rows, case["width"])
        if case["train"]:
            s["dx"], s["dy"] = _normal(g, rows, case["width"]), _normal(g, case["tokens"], case["width"])
        if own:
            import dense_fp32_matrix_f32_amd as sg
            s["routing"] = sg.Routing(s["offsets"], s["order"], s["position"])
    elif op == "experts":
        ids, _ = _router(g, case["tokens"], case["top"], case["experts"])
        s["offsets"], _, _ = _by_expert(ids, case["experts"])
        s["most"] = int(torch.diff(s["offsets"]).max())
        rows = case["tokens"] * case["top"]
        s["a"] = _normal(g, rows, case["k"])
        s["b"] = 0.02 * _normal(g, case["experts"], case["k"], case["n"])
        if case["train"]:
            s["dc"] = _normal(g, rows, case["n"])
    return s


# ---- one pass ---------------------------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import dense_fp32_matrix_f32_amd as sg
    case = s["case"]
    op = case["op"]
    if op == "w4":
        return sg.matmul_w4(s["a"], s["w"])
    if op == "w4_experts":
        return sg.matmul_w4(s["a"], s["w"], offsets=s["offsets"])
    if op == "sort":
        r = sg.sort_by_expert(s["ids"], case["experts"])
        return {"offsets": r.offsets, "order": r.order, "position": r.position}
    if op == "rows":
        out = {"rows": sg.gather_rows(s["x"], s["routing"]),
               "back": sg.combine_rows(s["y"], s["routing"], s["weights"])}
        if case["train"]:
            out["dy"], out["dweights"] = sg.combine_rows_grad(s["dy"], s["y"], s["routing"], s["weights"])
            out["dx"] = sg.combine_rows(s["dx"], s["routing"])
        return out
    out = {"c": sg.grouped_matmul(s["a"], s["b"], s["offsets"])}
    if case["train"]:
        out["da"] = sg.grouped_matmul(s["dc"], s["b"].transpose(1, 2), s["offsets"])
        out["db"] = sg.grouped_matmul_ta(s["a"], s["dc"], s["offsets"])
    return out


def _weights(codes, scales, zeros, k, group):
    """The weights that codes [.., ceil(k/2), n] stand for, in 32 bits."""
    q = torch.stack((codes & 15, codes >> 4), dim=-2).flatten(-3, -2)[..., :k, :].float()
    z = 8.0 if zeros is None else zeros.float().repeat_interleave(group, dim=-2)[..., :k, :]
    return (q - z) * scales.float().repeat_interleave(group, dim=-2)[..., :k, :]


def _row_experts(offsets, rows):
    """The expert of each row."""
    at = torch.arange(rows, device=offsets.device, dtype=torch.int32)
    return torch.searchsorted(offsets[1:].contiguous(), at, right=True)


def _slots(offsets, rows, most):
    """Each row's place where every expert has room for `most` rows."""
    e = _row_experts(offsets, rows)
    return e * most + torch.arange(rows, device=offsets.device) - offsets[e]


def _padded(x, slots, experts, most):
    out = torch.zeros((experts * most, x.shape[1]), device=x.device)
    return out.index_copy_(0, slots, x).view(experts, most, x.shape[1])


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "w4":
        return s["a"] @ _weights(s["codes"], s["scales"], s["zeros"], case["k"], case["group"])
    if op == "w4_experts":
        rows = s["a"].shape[0]
        if rows <= case["experts"]:  # fewer rows than experts: only the experts that the rows name
            e = _row_experts(s["offsets"], rows)
            w = _weights(s["codes"][e], s["scales"][e], None if s["zeros"] is None else s["zeros"][e], case["k"], case["group"])
            return torch.bmm(s["a"][:, None, :], w)[:, 0]
        w = _weights(s["codes"], s["scales"], s["zeros"], case["k"], case["group"])
        slots = _slots(s["offsets"], rows, s["most"])
        return torch.bmm(_padded(s["a"], slots, case["experts"], s["most"]), w).flatten(0, 1)[slots]
    if op == "sort":
        flat = s["ids"].reshape(-1)
        kept = (flat >= 0) & (flat < case["experts"])
        key = torch.where(kept, flat, case["experts"])
        order = torch.sort(key, stable=True).indices
        counts = torch.zeros(case["experts"] + 1, dtype=torch.int32, device=flat.device)
        counts.index_add_(0, key, torch.ones_like(key))
        ends = torch.cumsum(counts, 0, dtype=torch.int32)
        offsets = ends - counts
        at = torch.arange(flat.numel(), dtype=torch.int32, device=flat.device)
        position = torch.empty_like(flat)
        position[order] = at
        return {"offsets": offsets,
                "order": torch.where(at < offsets[-1], order.to(torch.int32), -1),
                "position": torch.where(kept, position, -1).view_as(s["ids"])}
    if op == "rows":
        top = case["top"]
        token = s["order"] // top
        place = s["position"].long()
        out = {"rows": s["x"][token], "back": (s["y"][place] * s["weights"][:, :, None]).sum(1)}
        if case["train"]:
            out["dy"] = s["dy"][token] * s["weights"].flatten()[s["order"].long()][:, None]
            out["dweights"] = (s["dy"][:, None, :] * s["y"][place]).sum(2)
            out["dx"] = s["dx"][place].sum(1)
        return out
    slots = _slots(s["offsets"], s["a"].shape[0], s["most"])
    a = _padded(s["a"], slots, case["experts"], s["most"])
    out = {"c": torch.bmm(a, s["b"]).flatten(0, 1)[slots]}
    if case["train"]:
        dc = _padded(s["dc"], slots, case["experts"], s["most"])
        out["da"] = torch.bmm(dc, s["b"].transpose(1, 2)).flatten(0, 1)[slots]
        out["db"] = torch.bmm(a.transpose(1, 2), dc)
    return out


# ---- what a pass cannot do without, and the definition in 64 bits -------------------------------


def _experts_met(case):
    """How many experts get a row, in the mean over routers without preference."""
    return case["experts"] * (1.0 - (1.0 - case["top"] / case["experts"]) ** case["tokens"])


def work(case):
    op = case["op"]
    if op in ("w4", "w4_experts"):
        n, k = case["n"], case["k"]
        rows = case["rows"] if op == "w4" else case["tokens"] * case["top"]
        groups = -(-k // case["group"])
        each = -(-k // 2) * n + groups * n * ((4 if case["scale"] == "f32" else 2) + (1 if case["zeros"] else 0))
        met = 1 if op == "w4" else _experts_met(case)
        return {"bytes": int(met * each + 4 * rows * (n + k)), "flops": 2 * rows * n * k}
    rows = case["tokens"] * case["top"]
    if op == "sort":
        return {"bytes": 12 * rows + 4 * (case["experts"] + 1), "flops": 0}
    if op == "rows":
        w = 4 * case["width"]
        there, back = (case["tokens"] + rows) * w, (rows + case["tokens"]) * w
        if not case["train"]:
            return {"bytes": there + back + 12 * rows, "flops": 2 * rows * case["width"]}
        grads = (case["tokens"] + 2 * rows) * w + (rows + case["tokens"]) * w
        return {"bytes": there + back + grads + 16 * rows, "flops": 6 * rows * case["width"]}
    n, k = case["n"], case["k"]
    once = 4 * rows * (n + k)
    weights = 4 * n * k
    if not case["train"]:
        return {"bytes": int(once + _experts_met(case) * weights), "flops": 2 * rows * n * k}
    # the product and both gradients share their inputs: each is read once
    return {"bytes": int(2 * once + _experts_met(case) * weights + case["experts"] * weights), "flops": 6 * rows * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("w4", "w4_experts"):
        k, group = case["k"], case["group"]

        def product(a, codes, scales, zeros):
            w = torch.empty((codes.shape[0] * 2, codes.shape[1]), dtype=torch.float64, device="cuda")
            w[0::2], w[1::2] = codes % 16, codes // 16
            w = w[:k]
            for i in range(scales.shape[0]):
                part = w[i * group:(i + 1) * group]
                part -= 8 if zeros is None else zeros[i].double()
                part *= scales[i].double()
            return a.double() @ w

        if op == "w4":
            return product(s["a"], s["codes"], s["scales"], s["zeros"])
        ends = s["offsets"].tolist()
        return torch.cat([product(s["a"][lo:hi], s["codes"][e], s["scales"][e], None if s["zeros"] is None else s["zeros"][e])
                          for e, (lo, hi) in enumerate(zip(ends, ends[1:]))])
    if op == "sort":
        ids = s["ids"].cpu().reshape(-1).tolist()
        lists = [[] for _ in range(case["experts"])]
        for f, e in enumerate(ids):
            if 0 <= e < case["experts"]:
                lists[e].append(f)
        offsets, order, position = [0], [], [-1] * len(ids)
        for one in lists:
            for f in one:
                position[f] = len(order)
                order.append(f)
            offsets.append(len(order))
        order += [-1] * (len(ids) - len(order))
        put = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"offsets": put(offsets), "order": put(order), "position": put(position).view_as(s["ids"])}
    if op == "rows":
        tokens, top = case["tokens"], case["top"]
        pos, w = s["position"].long(), s["weights"].double()
        rows = torch.empty((tokens * top, case["width"]), dtype=torch.float64, device="cuda")
        back = torch.zeros((tokens, case["width"]), dtype=torch.float64, device="cuda")
        out = {"rows": rows, "back": back}
        if case["train"]:
            out["dy"], out["dx"] = torch.empty_like(rows), torch.zeros_like(back)
            out["dweights"] = torch.empty_like(w)
        for j in range(top):
            rows[pos[:, j]] = s["x"].double()
            back += s["y"].double()[pos[:, j]] * w[:, j, None]
            if case["train"]:
                out["dy"][pos[:, j]] = s["dy"].double() * w[:, j, None]
                out["dweights"][:, j] = (s["dy"].double() * s["y"].double()[pos[:, j]]).sum(1)
                out["dx"] += s["dx"].double()[pos[:, j]]
        return out
    ends = s["offsets"].tolist()
    a, b = s["a"].double(), s["b"].double()
    spans = list(enumerate(zip(ends, ends[1:])))
    out = {"c": torch.cat([a[lo:hi] @ b[e] for e, (lo, hi) in spans])}
    if case["train"]:
        dc = s["dc"].double()
        out["da"] = torch.cat([dc[lo:hi] @ b[e].t() for e, (lo, hi) in spans])
        out["db"] = torch.stack([a[lo:hi].t() @ dc[lo:hi] for e, (lo, hi) in spans])
    return out
