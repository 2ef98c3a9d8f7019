"""Measured cases of the operators that stand around the quantised products:
the projection with per-row low-rank adapters (w4a16_gemm_lora) and the rows
of a mixture of experts (w4a16_expert_sort, _gather, _combine and gradients).

A case says what in real use it stands for beside its sizes. run() computes it
in its plain form (elementary torch operations in 32 bits, rounded once), or
with the library's own calls where `own` is true.
"""
import math

import torch

own = False

_NAMES = ("sort", "gather", "gather_grad", "combine", "combine_grad", "lora")


def _route(op, T, k, G, width, drop, name=None):
    c = {"op": op, "T": T, "k": k, "G": G, "width": width, "drop": drop}
    return {"name": name, **c} if name else c


def _lora(M, N, K, group, R, L, order, bare, name=None):
    c = {"op": "lora", "M": M, "N": N, "K": K, "group": group, "R": R, "L": L, "order": order, "bare": bare}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one decode step of 16 requests: latency of the smallest routing
        _route("sort", 16, 4, 8, 0, 0.0, "sort decode 16x4 G8"),
        # a long training batch, 8 of 128 experts, some padded tokens
        _route("sort", 65536, 8, 128, 0, 0.02, "sort long 65536x8 G128"),
        # the rows of a prefill batch brought into expert order
        _route("gather", 16384, 4, 64, 5120, 0.05, "gather long 16384x4x5120"),
        # the gradient of the same, at a ragged length with padding
        _route("gather_grad", 777, 3, 8, 4096, 0.1, "gather grad 777x3x4096"),
        # a ragged small batch with an odd width (rows not 16-byte aligned)
        _route("combine", 333, 3, 8, 1001, 0.0, "combine ragged 333x3x1001"),
        # the experts' outputs of a long prefill back in token order
        _route("combine", 16384, 8, 64, 4096, 0.0, "combine long 16384x8x4096"),
        # training at the grouped product's size (2048 rows, 8 experts, width 2048)
        _route("combine_grad", 1024, 2, 8, 2048, 0.0, "combine grad 1024x2x2048"),
        # training, long, with padded tokens
        _route("combine_grad", 8192, 8, 64, 4096, 0.03, "combine grad 8192x8x4096"),
        # the decode projection, one request with its adapter
        _lora(1, 17408, 5120, 128, 16, 8, "each", 0.0, "lora decode 1x17408x5120 r16"),
        # small-batch decode, every request with an adapter of its own
        _lora(16, 8192, 8192, 128, 16, 16, "each", 0.0, "lora batch 16x8192x8192 r16"),
        # the fused gate-up prefill, four requests one after the other, part of the rows without an adapter
        _lora(1322, 19456, 2560, 128, 64, 4, "runs", 0.1, "lora prefill 1322x19456x2560 r64"),
        # a tall-K projection at group 32, the rows of five adapters mixed
        _lora(333, 2560, 9728, 32, 24, 5, "mixed", 0.1, "lora ragged 333x2560x9728 g32 r24"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(_NAMES)
    if op == "lora":
        M, group = _log(rng, 1, 2048), rng.choice((128, 128, 32))
        N, K = _log(rng, 256, 19456), 128 * _log(rng, 2, 76)
        while M * N * K > 1322 * 19456 * 2560:
            M = max(1, M // 2)
        R, L = 8 * _log(rng, 1, 16), _log(rng, 1, 32)
        return _lora(M, N, K, group, R, L, rng.choice(("each", "runs", "mixed")), rng.choice((0.0, 0.1, 0.5)))
    G = _log(rng, 4, 256)
    k = min(rng.randint(1, 8), G)
    drop = rng.choice((0.0, 0.05, 0.3))
    if op == "sort":
        return _route(op, _log(rng, 1, 65536), k, G, 0, drop)
    T = _log(rng, 1, 16384)
    width = 128 * _log(rng, 1, 64) if op.startswith("gather") else _log(rng, 100, 8192)
    while T * k * width > 8192 * 8 * 4096:
        T = max(1, T // 2)
    return _route(op, T, k, G, width, drop)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(g, case):
    """Adapter of each row: one each in turn, runs of requests, or mixed; a share of bare rows without one."""
    M, L = case["M"], case["L"]
    if case["order"] == "each":
        ids = torch.arange(M, device="cuda") % L
        ids = (ids + torch.randint(0, L, (1,), generator=g, device="cuda")) % L
    elif case["order"] == "runs":
        cut = torch.rand(L, generator=g, device="cuda") + 0.2
        edge = (cut.cumsum(0) / cut.sum() * M).long()[:-1]
        ids = (torch.arange(M, device="cuda")[:, None] >= edge[None, :]).sum(1)
    else:
        ids = torch.randint(0, L, (M,), generator=g, device="cuda")
    if case["bare"] > 0 and case["order"] == "runs":
        ids[: int(M * case["bare"])] = -1
    elif case["bare"] > 0:
        ids[torch.rand(M, generator=g, device="cuda") < case["bare"]] = -1
    return ids.int()


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "lora":
        M, N, K, R, L, gs = (case[n] for n in ("M", "N", "K", "R", "L", "group"))
        s = {
            "op": "lora", "group": gs,
            "x": _randn(g, M, K).bfloat16(),
            "w": torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
            "s": (0.005 + 0.015 * torch.rand(N, K // gs, generator=g, device="cuda")).bfloat16(),
            "a": (_randn(g, L, R, K) * K ** -0.5).bfloat16(),
            "b": (_randn(g, L, N, R) * 0.1).bfloat16(),
            "scaling": 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda"),
            "ids": _rows(g, case),
            "y": torch.empty(M, N, dtype=torch.bfloat16, device="cuda"),
        }
        return s
    T, k, G, W = case["T"], case["k"], case["G"], case["width"]
    # a router's choice: experts of uneven popularity, softmax weights of the chosen ones, padded tokens dropped
    logits = _randn(g, T, G) + 0.5 * _randn(g, 1, G)
    top, ids = logits.topk(k, dim=1)
    ids = ids.int()
    ids[torch.rand(T, generator=g, device="cuda") < case["drop"]] = -1
    s = {"op": case["op"], "T": T, "k": k, "G": G, "ids": ids}
    if case["op"] == "sort":
        return s
    S = T * k
    s["order"], s["pos"], s["m_sizes"] = _sort(ids, G)
    s["weights"] = torch.softmax(top, dim=1)
    if case["op"] == "gather":
        s["x"] = _randn(g, T, W).bfloat16()
        s["out"] = torch.zeros(S, W, dtype=torch.bfloat16, device="cuda")   # rows behind the last one stay zero
    elif case["op"] == "gather_grad":
        s["dxs"] = _randn(g, S, W).bfloat16()
    else:
        s["z"] = _randn(g, S, W).bfloat16()
    if case["op"] == "combine_grad":
        s["dy"] = _randn(g, T, W).bfloat16()
        s["dz"] = torch.zeros(S, W, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _sort(ids, G):
    flat = ids.reshape(-1)
    valid = (flat >= 0) & (flat < G)
    key = torch.where(valid, flat, G).long()
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(flat.numel(), device=flat.device)
    pos = torch.where(valid, pos, -1)
    sizes = torch.zeros(G + 1, dtype=torch.int32, device=flat.device).index_add_(0, key, torch.ones_like(flat))
    return order.int(), pos.int().reshape(ids.shape), sizes[:G]


def _gather(x, pos):
    T, k = pos.shape
    S = T * k
    to = torch.where(pos >= 0, pos, S).reshape(-1).long()   # dropped slots go to one row behind
    out = torch.zeros(S + 1, x.shape[1], dtype=x.dtype, device=x.device)
    out[to] = x[:, None, :].expand(T, k, x.shape[1]).reshape(S, -1)
    return out[:S]


def _weighted(z, pos, w):
    rows = z[pos.clamp(min=0).long()].float()                # [T, k, width]
    rows = torch.where((pos >= 0)[:, :, None], rows, 0.0)
    if w is not None:
        rows = rows * w[:, :, None]
    return rows.sum(1).bfloat16()


def _combine_grad(dy, z, pos, w):
    T, k = pos.shape
    keep = pos >= 0
    S = T * k
    d = dy.float()
    to = torch.where(keep, pos, S).reshape(-1).long()
    dz = torch.zeros(S + 1, dy.shape[1], dtype=dy.dtype, device=dy.device)
    dz[to] = (d[:, None, :] * w[:, :, None]).bfloat16().reshape(S, -1)
    rows = z[pos.clamp(min=0).long()].float()
    dw = torch.where(keep, (rows * d[:, None, :]).sum(2), 0.0)
    return dz[:S], dw


def _dequant(w, s, gs):
    q = torch.stack((w & 15, w >> 4), dim=2).reshape(w.shape[0], -1).float() - 8.0
    return (q.reshape(q.shape[0], -1, gs) * s.float()[:, :, None]).reshape(q.shape)


def _lora_plain(t):
    x = t["x"].float()
    L, R, K = t["a"].shape
    y = x @ _dequant(t["w"], t["s"], t["group"]).t()
    h = (x @ t["a"].float().reshape(L * R, K).t()).reshape(-1, L, R)
    mine = (t["ids"][:, None] == torch.arange(L, device=x.device)[None, :]).float() * t["scaling"][None, :]
    h = (h * mine[:, :, None]).reshape(-1, L * R)
    y = y + h @ t["b"].float().permute(0, 2, 1).reshape(L * R, -1)
    return y.bfloat16()


def run(state):
    t, op = state, state["op"]
    if own:
        import bf16_activation_quantized_amd as w4
        if op == "sort":
            return w4.w4a16_expert_sort(t["ids"], t["G"])
        if op == "gather":
            return w4.w4a16_expert_gather(t["x"], t["pos"], xs=t["out"])
        if op == "gather_grad":
            return w4.w4a16_expert_gather_grad(t["dxs"], t["pos"])
        if op == "combine":
            return w4.w4a16_expert_combine(t["z"], t["pos"], t["weights"])
        if op == "combine_grad":
            return w4.w4a16_expert_combine_grad(t["dy"], t["z"], t["pos"], t["weights"], dz=t["dz"])
        return w4.w4a16_gemm_lora(t["x"], t["w"], t["s"], t["a"], t["b"], t["ids"], scaling=t["scaling"], y=t["y"],
                                  group_size=t["group"])
    if op == "sort":
        return _sort(t["ids"], t["G"])
    if op == "gather":
        return _gather(t["x"], t["pos"])
    if op == "gather_grad":
        return _weighted(t["dxs"], t["pos"], None)
    if op == "combine":
        return _weighted(t["z"], t["pos"], t["weights"])
    if op == "combine_grad":
        return _combine_grad(t["dy"], t["z"], t["pos"], t["weights"])
    return _lora_plain(t)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "lora":
        M, N, K, R, gs = (case[n] for n in ("M", "N", "K", "R", "group"))
        present = min(case["L"], max(1, int(M * (1.0 - case["bare"]))))
        byts = N * K // 2 + N * (K // gs) * 2 + M * K * 2 + M * N * 2 + present * R * (K + N) * 2 + 4 * M
        return {"bytes": byts, "flops": 2 * M * N * K + 2 * int(M * (1.0 - case["bare"])) * R * (K + N)}
    T, k, W = case["T"], case["k"], case["width"]
    S = T * k
    kept = int(S * (1.0 - case["drop"]))
    if op == "sort":
        return {"bytes": 12 * S + 4 * case["G"], "flops": 0}
    if op == "gather":
        return {"bytes": 2 * W * (T + kept) + 4 * S, "flops": 0}
    if op == "gather_grad":
        return {"bytes": 2 * W * (T + kept) + 4 * S, "flops": W * kept}
    if op == "combine":
        return {"bytes": 2 * W * (T + kept) + 8 * S, "flops": 2 * W * kept}
    return {"bytes": 2 * W * (T + 2 * kept) + 12 * S, "flops": 3 * W * kept}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    t = prepare(case, seed)
    op = case["op"]
    if op == "lora":
        x = t["x"].double()
        N, K = case["N"], case["K"]
        y = torch.empty(case["M"], N, dtype=torch.float64, device="cuda")
        for n0 in range(0, N, 4096):   # the product in column blocks: the weights in 64 bits are large
            w = t["w"][n0:n0 + 4096].to(torch.int16)
            d = torch.empty(w.shape[0], K, dtype=torch.float64, device="cuda")
            d[:, 0::2] = (w % 16).double() - 8
            d[:, 1::2] = torch.div(w, 16, rounding_mode="floor").double() - 8
            d *= t["s"][n0:n0 + 4096].double().repeat_interleave(case["group"], dim=1)
            y[:, n0:n0 + 4096] = x @ d.t()
        for a in range(case["L"]):
            rows = (t["ids"] == a).nonzero().flatten()
            if len(rows):
                h = x[rows] @ t["a"][a].double().t()
                y[rows] += t["scaling"][a].double() * (h @ t["b"][a].double().t())
        return y
    if op == "sort":
        e = t["ids"].flatten().tolist()
        G = case["G"]
        bins = [[] for _ in range(G + 1)]
        for slot, i in enumerate(e):
            bins[i if 0 <= i < G else G].append(slot)
        order = [slot for b in bins for slot in b]
        pos = [-1] * len(e)
        for p, slot in enumerate(order[: len(e) - len(bins[G])]):
            pos[slot] = p
        T, k = t["ids"].shape
        return (torch.tensor(order, dtype=torch.int32), torch.tensor(pos, dtype=torch.int32).reshape(T, k),
                torch.tensor([len(b) for b in bins[:G]], dtype=torch.int32))
    T, k, W = case["T"], case["k"], case["width"]
    kept = int(t["m_sizes"].sum())
    slot = t["order"][:kept].long()          # the slot that each sorted row holds
    token = torch.div(slot, k, rounding_mode="floor")
    if op == "gather":
        out = torch.zeros(T * k, W, dtype=torch.float64, device="cuda")
        out[:kept] = t["x"][token].double()
        return out
    if op in ("gather_grad", "combine"):
        rows = t["dxs" if op == "gather_grad" else "z"][:kept]
        w = t["weights"].flatten()[slot].double()
        y = torch.zeros(T, W, dtype=torch.float64, device="cuda")
        for r0 in range(0, kept, 16384):
            part = rows[r0:r0 + 16384].double()
            if op == "combine":
                part = part * w[r0:r0 + 16384, None]
            y.index_add_(0, token[r0:r0 + 16384], part)
        return y
    w = t["weights"].flatten()[slot].double()
    dz = torch.zeros(T * k, W, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    for r0 in range(0, kept, 16384):
        r1 = min(kept, r0 + 16384)
        d = t["dy"][token[r0:r1]].double()
        dz[r0:r1] = d * w[r0:r1, None]
        dw[slot[r0:r1]] = (d * t["z"][r0:r1].double()).sum(1)
    return dz, dw.reshape(T, k)
