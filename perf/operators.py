"""Cases for the products whose rows choose their matrix: routing rows to groups
and back, the groups' products with their gradients, and low-rank adapters of
many requests beside a shared projection.

``run`` computes a case with elementary torch operations in 32 bits (``own``
false) or with the library's operators (``own`` true).
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # One decoding step of a mixture-of-experts block: few tokens, many
        # experts.  Latency counts.
        dict(name="route_decode", op="route", dtype="bf16", tokens=64, choices=8, groups=128,
             cols=2048, skew=0.3, drop=0.0),
        # The rows of a prefill or training batch sorted by expert.
        dict(name="route_batch", op="route", dtype="bf16", tokens=8192, choices=8, groups=64,
             cols=2048, skew=0.5, drop=0.0),
        # The gradient of that gather, ragged: rows that are no whole number
        # of 16-byte words, and tokens that another rank's experts take.
        dict(name="gather_grad_ragged", op="gather_grad", dtype="f16", tokens=4099, choices=6,
             groups=60, cols=1410, skew=0.5, drop=0.2),
        # The experts' rows of a batch added up by their router weights.
        dict(name="combine_batch", op="combine", dtype="bf16", tokens=8192, choices=8, groups=64,
             cols=2048, skew=0.5, drop=0.0),
        # Its gradient, in single precision.
        dict(name="combine_grad_f32", op="combine_grad", dtype="f32", tokens=4096, choices=2,
             groups=16, cols=4096, skew=0.5, drop=0.05),
        # The experts' products of a decoding step: a few rows per expert, so
        # the time is that of reading the weights.
        dict(name="experts_decode", op="grouped", dtype="bf16", tokens=64, choices=8, groups=128,
             K=2048, N=1536, skew=0.3, drop=0.0, trans=False, out="bf16"),
        # The experts' products of a large batch (the largest case).
        dict(name="experts_batch", op="grouped", dtype="bf16", tokens=8192, choices=8, groups=64,
             K=2048, N=1536, skew=0.5, drop=0.0, trans=False, out="bf16"),
        # The gradient of such a product's input: the weights enter
        # transposed; skewed groups and odd row counts.
        dict(name="experts_input_grad", op="grouped", dtype="f16", tokens=10007, choices=2,
             groups=16, K=1408, N=4096, skew=1.0, drop=0.1, trans=True, out="f16"),
        # The gradient of the weights, kept in fp32 as an optimizer wants it.
        dict(name="experts_weight_grad", op="wgrad", dtype="bf16", tokens=8192, choices=4,
             groups=32, K=2048, N=1536, skew=0.5, drop=0.0, out="f32"),
        # A decoding step of many requests, each with its own adapter.
        dict(name="adapter_decode", op="adapter", dtype="bf16", rows=32, K=4096, N=4096, rank=16,
             adapters=32, requests=32, none=0.1, trans=True, out="bf16"),
        # Prompts of a few requests at once: long runs of rows of one adapter.
        dict(name="adapter_prompts", op="adapter", dtype="bf16", rows=4096, K=4096, N=4096,
             rank=64, adapters=8, requests=11, none=0.2, trans=True, out="bf16"),
        # Short and long requests mixed, at sizes that fill no tile.
        dict(name="adapter_mixed", op="adapter", dtype="f16", rows=333, K=2056, N=5000, rank=12,
             adapters=20, requests=70, none=0.25, trans=False, out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _length(rng, lo, hi):
    """A row length: mostly multiples of 8, sometimes odd."""
    n = _log(rng, lo, hi)
    n = n if rng.random() < 0.25 else max(8, n // 8 * 8)
    return n + 8 if n == 3072 else n


def draw(rng):
    op = rng.choice(["route", "gather_grad", "combine", "combine_grad", "grouped", "grouped",
                     "wgrad", "adapter", "adapter"])
    big = [work(c) for c in listed() if c["op"] in (op, "grouped" if op == "wgrad" else op)]
    most = {k: max(w[k] for w in big) for k in ("bytes", "flops")}
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    while True:
        case = dict(op=op, dtype=dtype)
        if op == "adapter":
            rows = _log(rng, 1, 4096)
            case.update(rows=rows, K=_length(rng, 256, 6000), N=_length(rng, 256, 6000),
                        rank=rng.choice([4, 8, 12, 16, 32, 64]), adapters=_log(rng, 1, 64),
                        requests=_log(rng, 1, min(rows, 128)), none=rng.choice([0.0, 0.25]),
                        trans=rng.random() < 0.5, out=rng.choice([dtype, "f32"]))
        else:
            choices = rng.choice([1, 2, 4, 6, 8])
            case.update(tokens=_log(rng, 1, 8192), choices=choices,
                        groups=_log(rng, max(choices, 4), 128),
                        skew=rng.choice([0.0, 0.5, 1.0]), drop=rng.choice([0.0, 0.0, 0.2]))
            if op in ("grouped", "wgrad"):
                case.update(K=_length(rng, 256, 4096), N=_length(rng, 256, 4096),
                            out=rng.choice([dtype, "f32"]))
                if op == "grouped":
                    case.update(trans=rng.random() < 0.5)
            else:
                case.update(cols=_length(rng, 256, 4096))
        w = work(case)
        # matrix products in fp32 run at about a sixteenth of the 16-bit rate
        cost = 16 if dtype == "f32" else 1
        if w["bytes"] <= most["bytes"] and w["flops"] * cost <= most["flops"] + 1e9:
            return case


def _ids(case, gen):
    """tokens x choices distinct group ids per token, group g chosen in
    proportion to (g + 1)^-skew; a share `drop` of the entries is -1 (experts
    that live elsewhere)."""
    T, k, G = case["tokens"], case["choices"], case["groups"]
    rank = torch.arange(1, G + 1, device="cuda", dtype=torch.float32)
    noise = -torch.log(-torch.log(torch.rand(T, G, device="cuda", generator=gen) * 0.999998 + 1e-6))
    scores, ids = torch.topk(noise - case["skew"] * torch.log(rank), k, dim=1)
    ids = ids.to(torch.int32)
    if case["drop"]:
        gone = torch.rand(T, k, device="cuda", generator=gen) < case["drop"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.contiguous(), torch.softmax(scores, dim=1).contiguous()


def _normal(shape, dtype, gen, scale=1.0):
    x = torch.empty(shape, device="cuda", dtype=TYPES[dtype])
    x.normal_(0.0, scale, generator=gen)
    return x


def _sorted_rows(ids, groups):
    """offsets (G + 1), order (R) and position (T x k) of a stable sort of the
    entries by group, entries of no group last."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < groups), flat, torch.full_like(flat, groups))
    at = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key[at], torch.arange(groups + 1, device=ids.device))
    row = torch.empty_like(at)
    row[at] = torch.arange(at.numel(), device=ids.device)
    position = torch.where(key < groups, row, torch.full_like(row, -1)).reshape(ids.shape)
    order = torch.where(key[at] < groups, at, torch.full_like(at, -1))
    return offsets.int(), order.int(), position.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dtype = case["op"], case["dtype"]
    state = {"case": dict(case)}
    if op == "adapter":
        T, K, N, r, L = (case[n] for n in ("rows", "K", "N", "rank", "adapters"))
        state["x"] = _normal((T, K), dtype, gen)
        if case["trans"]:  # a linear layer's weight: N x K
            state["w"] = _normal((N, K), dtype, gen, K ** -0.5).t()
        else:
            state["w"] = _normal((K, N), dtype, gen, K ** -0.5)
        state["a"] = _normal((L, r, K), dtype, gen, K ** -0.5)
        state["b"] = _normal((L, N, r), dtype, gen, r ** -0.5)
        state["scales"] = torch.rand(L, device="cuda", generator=gen) * 1.5 + 0.25
        # requests are runs of rows of random lengths, each with one adapter
        cuts = torch.sort(torch.rand(case["requests"], device="cuda", generator=gen)).values
        run_of = torch.searchsorted(cuts, (torch.arange(T, device="cuda") + 0.5) / T)
        if T == case["requests"]:  # a decoding step: one row each
            run_of = torch.arange(T, device="cuda")
        pick = torch.randint(0, L, (case["requests"] + 1,), device="cuda", generator=gen)
        if L >= case["requests"]:  # an adapter of its own for each
            pick = torch.randperm(L + 1, device="cuda", generator=gen)[:case["requests"] + 1] % L
        bare = torch.rand(pick.numel(), device="cuda", generator=gen) < case["none"]
        pick = torch.where(bare, torch.full_like(pick, -1), pick)
        state["ids"] = pick[run_of].to(torch.int32).contiguous()
        return state
    ids, weights = _ids(case, gen)
    T, k = ids.shape
    if op == "route":
        state["ids"] = ids
        state["x"] = _normal((T, case["cols"]), dtype, gen)
        return state
    offsets, order, position = _sorted_rows(ids, case["groups"])
    state["offsets"] = offsets
    if op == "grouped":
        state["a"] = _normal((T * k, case["K"]), dtype, gen)
        G, K, N = case["groups"], case["K"], case["N"]
        if case["trans"]:
            state["b"] = _normal((G, N, K), dtype, gen, K ** -0.5).transpose(1, 2)
        else:
            state["b"] = _normal((G, K, N), dtype, gen, K ** -0.5)
    elif op == "wgrad":
        state["a"] = _normal((T * k, case["K"]), dtype, gen)
        state["dc"] = _normal((T * k, case["N"]), dtype, gen)
    else:
        state.update(ids=ids, order=order, position=position, weights=weights)
        if op == "combine":
            state["ys"] = _normal((T * k, case["cols"]), dtype, gen)
        elif op == "combine_grad":
            state["ys"] = _normal((T * k, case["cols"]), dtype, gen)
            state["dy"] = _normal((T, case["cols"]), dtype, gen)
        else:
            state["dxs"] = _normal((T * k, case["cols"]), dtype, gen)
    return state


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import persistent_stream_tiling_amd as gsk
    c = s["case"]
    op = c["op"]
    if op == "route":
        r = gsk.route_rows(s["ids"], c["groups"])
        return {"offsets": r.offsets, "order": r.order, "position": r.position,
                "xs": gsk.gather_rows(s["x"], r)}
    if op == "grouped":
        return gsk.grouped_matmul(s["a"], s["b"], s["offsets"], out_dtype=TYPES[c["out"]])
    if op == "wgrad":
        return gsk.grouped_matmul_wgrad(s["a"], s["dc"], s["offsets"], out_dtype=TYPES[c["out"]])
    if op == "adapter":
        return gsk.adapter_matmul(s["x"], s["w"], s["a"], s["b"], s["ids"], s["scales"],
                                  out_dtype=TYPES[c["out"]])
    r = gsk.Routing(s["offsets"], s["order"], s["position"])
    if op == "combine":
        return gsk.combine_rows(s["ys"], s["weights"], r)
    if op == "combine_grad":
        dys, dw = gsk.combine_rows_backward(s["dy"], s["ys"], s["weights"], r)
        return {"dys": dys, "dweights": dw}
    return gsk.gather_rows_backward(s["dxs"], r)


def _run_plain(s):
    c = s["case"]
    op, dtype = c["op"], TYPES[c["dtype"]]
    if op == "route":
        offsets, order, position = _sorted_rows(s["ids"], c["groups"])
        x = s["x"].float()
        at = torch.clamp(order.long(), min=0) // c["choices"]
        xs = x[at] * (order >= 0).float()[:, None]
        return {"offsets": offsets, "order": order, "position": position, "xs": xs.to(dtype)}
    if op == "grouped":
        a, b, out = s["a"], s["b"], TYPES[c["out"]]
        bounds = s["offsets"].tolist()
        res = torch.zeros(a.shape[0], b.shape[2], device=a.device, dtype=out)
        for g in range(b.shape[0]):
            lo, hi = bounds[g], bounds[g + 1]
            if hi > lo:
                res[lo:hi] = torch.mm(a[lo:hi].float(), b[g].float()).to(out)
        return res
    if op == "wgrad":
        a, dc, out = s["a"], s["dc"], TYPES[c["out"]]
        bounds = s["offsets"].tolist()
        G = len(bounds) - 1
        res = torch.zeros(G, a.shape[1], dc.shape[1], device=a.device, dtype=out)
        for g in range(G):
            lo, hi = bounds[g], bounds[g + 1]
            if hi > lo:
                res[g] = torch.mm(a[lo:hi].float().t(), dc[lo:hi].float()).to(out)
        return res
    if op == "adapter":
        x, ids, L = s["x"].float(), s["ids"].long(), s["a"].shape[0]
        y = torch.mm(x, s["w"].float())
        has = (ids >= 0) & (ids < L)
        for g in torch.unique(ids[has]).tolist():
            rows = (ids == g).nonzero().squeeze(1)
            h = torch.mm(x[rows], s["a"][g].float().t()) * s["scales"][g]
            y[rows] += torch.mm(h, s["b"][g].float().t())
        return y.to(TYPES[c["out"]])
    T, k = s["position"].shape
    pos = torch.clamp(s["position"].long(), min=0)
    live = (s["position"] >= 0).float()
    if op == "combine":
        w = s["weights"] * live
        y = torch.zeros(T, c["cols"], device=w.device)
        for j in range(k):
            y += w[:, j:j + 1] * s["ys"][pos[:, j]].float()
        return y.to(dtype)
    if op == "combine_grad":
        dy = s["dy"].float()
        w = s["weights"]
        dw = torch.zeros_like(w)
        for j in range(k):
            dw[:, j] = (dy * s["ys"][pos[:, j]].float()).sum(1) * live[:, j]
        at = torch.clamp(s["order"].long(), min=0)
        wr = w.reshape(-1)[at] * (s["order"] >= 0).float()
        dys = (wr[:, None] * dy[at // k]).to(dtype)
        return {"dys": dys, "dweights": dw}
    dx = torch.zeros(T, c["cols"], device=pos.device)
    for j in range(k):
        dx += live[:, j:j + 1] * s["dxs"][pos[:, j]].float()
    return dx.to(dtype)


def exact(case, seed):
    """The definitions entry by entry of the sorted order, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "adapter":
        x, L = s["x"].double(), s["a"].shape[0]
        y = x @ s["w"].double()
        for g in range(L):
            mine = (s["ids"] == g).double()[:, None]
            if bool(mine.any()):
                y = y + float(s["scales"][g]) * (((mine * x) @ s["a"][g].double().T) @
                                                 s["b"][g].double().T)
        return y
    if op == "route":
        ids = s["ids"].cpu().reshape(-1).tolist()
        G, k = case["groups"], case["choices"]
        buckets = [[] for _ in range(G)]
        for i, g in enumerate(ids):
            if 0 <= g < G:
                buckets[g].append(i)
        order = [i for b in buckets for i in b]
        offsets, position = [0], [-1] * len(ids)
        for b in buckets:
            offsets.append(offsets[-1] + len(b))
        for r, i in enumerate(order):
            position[i] = r
        xs = torch.zeros(len(ids), case["cols"], device="cuda", dtype=torch.float64)
        xs[:len(order)] = s["x"].double()[torch.tensor(order, device="cuda", dtype=torch.long) // k]
        order += [-1] * (len(ids) - len(order))
        whole = dict(device="cuda", dtype=torch.int32)
        return {"offsets": torch.tensor(offsets, **whole), "order": torch.tensor(order, **whole),
                "position": torch.tensor(position, **whole).reshape(-1, k), "xs": xs}
    off = [int(v) for v in s["offsets"].cpu()]
    if op == "grouped":
        parts = [s["a"][lo:hi].double() @ s["b"][g].double()
                 for g, (lo, hi) in enumerate(zip(off, off[1:]))]
        parts.append(torch.zeros(s["a"].shape[0] - off[-1], case["N"], device="cuda",
                                 dtype=torch.float64))
        return torch.cat(parts)
    if op == "wgrad":
        return torch.stack([s["a"][lo:hi].double().T @ s["dc"][lo:hi].double()
                            for lo, hi in zip(off, off[1:])])
    T, k = s["ids"].shape
    order = s["order"][:off[-1]].long()
    tok = order // k
    if op in ("combine", "gather_grad"):
        src = s["ys"] if op == "combine" else s["dxs"]
        rows = src[:off[-1]].double()
        if op == "combine":
            rows = rows * s["weights"].double().reshape(-1)[order][:, None]
        out = torch.zeros(T, case["cols"], device="cuda", dtype=torch.float64)
        return out.index_add_(0, tok, rows)
    dy = s["dy"].double()
    w = s["weights"].double().reshape(-1)
    dys = torch.zeros(T * k, case["cols"], device="cuda", dtype=torch.float64)
    dys[:off[-1]] = dy[tok] * w[order][:, None]
    dw = torch.zeros(T * k, device="cuda", dtype=torch.float64)
    dw[order] = (dy[tok] * s["ys"][:off[-1]].double()).sum(1)
    return {"dys": dys, "dweights": dw.reshape(T, k)}


def _present(n, among, skew=0.0):
    """Expected number of distinct values among n picks of `among`, the value
    g in proportion to (g + 1)^-skew."""
    p = [(g + 1.0) ** -skew for g in range(among)]
    total = sum(p)
    return sum(1.0 - (1.0 - q / total) ** n for q in p)


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "adapter":
        T, K, N, r, L = (case[n] for n in ("rows", "K", "N", "rank", "adapters"))
        runs = case["requests"] * (1 - case["none"])
        here = min(L, runs) if L >= case["requests"] else _present(runs, L)
        return {"bytes": e * (T * K + K * N + here * r * (K + N)) + 4 * (T + L) +
                SIZE[case["out"]] * T * N,
                "flops": 2.0 * T * K * N + 2.0 * T * (1 - case["none"]) * r * (K + N)}
    T, k, G = case["tokens"], case["choices"], case["groups"]
    R = T * k
    live = R * (1 - case["drop"])
    if op in ("grouped", "wgrad"):
        K, N, eo = case["K"], case["N"], SIZE[case["out"]]
        flops = 2.0 * live * K * N
        if op == "wgrad":
            return {"bytes": e * live * (K + N) + eo * G * K * N + 4 * (G + 1), "flops": flops}
        return {"bytes": e * (live * K + _present(live, G, case["skew"]) * K * N) + eo * R * N +
                4 * (G + 1), "flops": flops}
    H = case["cols"]
    if op == "route":
        return {"bytes": e * (T + R) * H + 12 * R + 4 * (G + 1), "flops": 0.0}
    if op == "combine":
        return {"bytes": e * (live + T) * H + 8 * R, "flops": 2.0 * live * H}
    if op == "combine_grad":
        return {"bytes": e * (live + T + R) * H + 16 * R, "flops": 3.0 * live * H}
    return {"bytes": e * (live + T) * H + 4 * R, "flops": 1.0 * live * H}
