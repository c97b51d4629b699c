"""Cases of the MoE layer's expert operators: routing by groups, the expert map, the experts' products and the
shared projection with low-rank adapters, in plain form (`own` false) and as the library's calls (`own` true)."""

import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one decoded token: 256 experts in 8 groups, sigmoid scores with a balance bias; latency counts
        dict(name="route T1", op="route", T=1, E=256, k=8, n_group=8, topk_group=4, group_top=2, scores="sigmoid", bias=True,
             renorm=True),
        # a prefill batch through the same router
        dict(name="route T8192", op="route", T=8192, E=256, k=8, n_group=8, topk_group=4, group_top=2, scores="sigmoid",
             bias=True, renorm=True),
        # a decode batch padded from 59 to 64 tokens: the padding's ids name no expert
        dict(name="map T64", op="map", T=64, E=256, k=8, block=1, drop=5, skew=0.5),
        # a prefill batch, segments padded to tiles of 128 rows
        dict(name="map T8192", op="map", T=8192, E=256, k=8, block=128, drop=0, skew=0.5),
        # one decoded token: 8 experts' gate and up weights
        dict(name="gate_up T1", op="expert", T=1, E=64, k=8, K=6144, N=4096, act="swiglu", gather=True, skew=0.0),
        # a decode batch: nearly every expert is read for one to a few rows
        dict(name="gate_up T64", op="expert", T=64, E=256, k=8, K=6144, N=4096, act="swiglu", gather=True, skew=0.5),
        # a prefill batch, uneven experts: the largest product
        dict(name="gate_up T8192", op="expert", T=8192, E=256, k=8, K=6144, N=4096, act="swiglu", gather=True, skew=0.5),
        # an odd verify batch of a ragged layer: down projection of rows that lie expert after expert
        dict(name="down T37 ragged", op="expert", T=37, E=168, k=6, K=1032, N=2056, act="none", gather=False, skew=0.5),
        # a middle batch's down projection
        dict(name="down T2048", op="expert", T=2048, E=256, k=8, K=2048, N=6144, act="none", gather=False, skew=0.5),
        # one decoded token with its adapter through the shared expert's gate and up projection
        dict(name="adapter T1", op="adapter", T=1, K=6144, N=4096, R=16, L=16, act="swiglu", requests=1),
        # a decode batch, nearly each token a request with an adapter of its own, down projection
        dict(name="adapter T64", op="adapter", T=64, K=2048, N=6144, R=16, L=64, act="none", requests=64),
        # prefill chunks of 11 requests over 8 adapters, gate and up projection
        dict(name="adapter T4096", op="adapter", T=4096, K=6144, N=4096, R=64, L=8, act="swiglu", requests=11),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "map", "expert", "expert", "adapter"])
    T = _log(rng, 1, 8192)
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8, 16])
        E = n_group * _log(rng, 4, 256 // n_group)
        topk_group = rng.randint((n_group + 1) // 2, n_group)
        k = rng.randint(1, min(16, E // n_group * topk_group))
        return dict(op=op, T=T, E=E, k=k, n_group=n_group, topk_group=topk_group, group_top=rng.choice([1, 2]),
                    scores=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.7, renorm=rng.random() < 0.7)
    if op == "map":
        E = _log(rng, 4, 512)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), block=rng.choice([1, 1, 8, 16, 128]),
                    drop=rng.randint(0, T // 4), skew=rng.choice([0.0, 0.5, 1.0]))
    act = rng.choice(["none", "swiglu"])
    K = _log(rng, 256, 6144 if act == "swiglu" else 2048, 8)  # gate and up, or down
    N = _log(rng, 128, 2048, 8) * 2 if act == "swiglu" else _log(rng, 256, 6144, 8)
    if op == "expert":
        E = _log(rng, 8, 256)
        return dict(op=op, T=T, E=E, k=rng.randint(1, 8), K=K, N=N, act=act, gather=rng.random() < 0.5,
                    skew=rng.choice([0.0, 0.5]))
    T = _log(rng, 1, 4096)
    return dict(op=op, T=T, K=K, N=N, R=rng.choice([8, 16, 32, 64]), L=_log(rng, 1, 64), act=act, requests=rng.randint(1, min(T, 64)))


def _ids(c, g):
    """k distinct experts a token, some experts more popular than others."""
    T, E, k = c["T"], c["E"], c["k"]
    popular = torch.randn(E, generator=g, device=DEV) * c["skew"]
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    ids = torch.topk(popular + noise, k, dim=1).indices.to(torch.int32)
    if c.get("drop"):
        ids[T - c["drop"]:] = -1
    return ids


def _bf16(g, std, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16) * std


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case=c)
    if c["op"] == "route":
        s["logits"] = torch.randn(c["T"], c["E"], generator=g, device=DEV) * 1.5
        s["bias"] = torch.randn(c["E"], generator=g, device=DEV) * 0.1 if c["bias"] else None
    elif c["op"] == "map":
        s["ids"] = _ids(c, g)
    elif c["op"] == "expert":
        T, E, k, K, N = c["T"], c["E"], c["k"], c["K"], c["N"]
        ids = _ids(c, g)
        order = torch.argsort(ids.reshape(-1), stable=True)
        s["counts"] = torch.bincount(ids.reshape(-1), minlength=E).to(torch.int32)
        s["offsets"] = torch.cat([s["counts"].new_zeros(1), torch.cumsum(s["counts"], 0, dtype=torch.int32)])
        s["row_token"] = (order // k).to(torch.int32) if c["gather"] else None
        s["expert"] = ids.reshape(-1)[order].to(torch.int64)
        s["widest"] = int(s["counts"].max().item())
        s["x"] = _bf16(g, 1.0, T if c["gather"] else T * k, K)
        s["w"] = _bf16(g, 0.02, E, N, K)
    else:
        T, K, N, R, L = c["T"], c["K"], c["N"], c["R"], c["L"]
        s["x"] = _bf16(g, 1.0, T, K)
        s["w"] = _bf16(g, 0.02, N, K)
        s["a"] = _bf16(g, 1.0 / math.sqrt(K), L, R, K)
        s["b"] = _bf16(g, 0.05, L, N, R)
        s["scale"] = torch.rand(L, generator=g, device=DEV) + 0.5
        # requests' tokens follow one another; one request in eight has no adapter
        of = torch.randint(0, L, (c["requests"],), generator=g, device=DEV)
        of = torch.where(torch.rand(c["requests"], generator=g, device=DEV) < 0.125, -1, of)
        s["ids"] = of[torch.arange(T, device=DEV) * c["requests"] // T].to(torch.int32)
    return s


# ------------------------------------------------------------------ plain forms


def _route_plain(c, logits, bias):
    T, E, G = c["T"], c["E"], c["n_group"]
    z = logits.double()  # choices next to a border, so in 64 bits
    s = torch.sigmoid(z) if c["scores"] == "sigmoid" else torch.softmax(z, dim=1)
    key = z if bias is None else s + bias.double()  # without a bias the order is that of the logits
    v = s if bias is None else key
    top = v.reshape(T, G, E // G).sort(dim=2, descending=True).values[:, :, : c["group_top"]].sum(2)
    chosen = top.sort(dim=1, descending=True, stable=True).indices[:, : c["topk_group"]]
    inside = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, chosen, True)
    key = key.masked_fill(~inside.repeat_interleave(E // G, dim=1), -math.inf)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, : c["k"]]
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(ids=ids.to(torch.int32), w=(2.5 * w).float())


def _rows_needed(c):
    n = c["T"] * c["k"]
    return n + min(c["E"], n) * (c["block"] - 1)


def _map_plain(c, ids):
    T, E, k, block = c["T"], c["E"], c["k"], c["block"]
    e = torch.where((ids >= 0) & (ids < E), ids, E).reshape(-1).to(torch.int64)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=e.device).scatter_add_(0, e, torch.ones_like(e))
    sizes = (counts + block - 1) // block * block
    ends = torch.cumsum(sizes, 0)
    order = torch.argsort(e, stable=True)
    se = e[order]
    first = torch.cumsum(counts, 0) - counts
    row = ends[se] - sizes[se] + torch.arange(T * k, device=e.device) - first[se]
    row = torch.where(se < E, row, -1)
    row_map = torch.empty_like(row).scatter_(0, order, row)
    n = _rows_needed(c)
    row_token = torch.full((n + 1,), -1, dtype=torch.int64, device=e.device)
    row_token[torch.where(row < 0, n, row)] = torch.where(row < 0, -1, order // k)
    return dict(row_map=row_map.reshape(T, k).to(torch.int32), row_token=row_token[:n].to(torch.int32),
                offsets=torch.cat([ends.new_zeros(1), ends[:E]]).to(torch.int32), counts=counts[:E].to(torch.int32))


def _act_plain(y, act):
    if act == "none":
        return y.to(torch.bfloat16)
    gate, up = y.chunk(2, dim=-1)
    return (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)


def _expert_plain(s, c):
    x = (s["x"] if s["row_token"] is None else s["x"][s["row_token"].long()]).float()
    e = s["expert"]
    if len(e) * 4 <= c["E"]:  # few rows: each row's own weights
        return _act_plain((s["w"][e].float() @ x[:, :, None])[:, :, 0], c["act"])
    at = torch.arange(len(e), device=e.device) - s["offsets"][e].long()
    padded = torch.zeros(c["E"], s["widest"], c["K"], device=x.device)
    padded[e, at] = x
    return _act_plain(torch.bmm(padded, s["w"].float().transpose(1, 2))[e, at], c["act"])


def _adapter_plain(s, c):
    T, L, R = c["T"], c["L"], c["R"]
    x = s["x"].float()
    mine = (s["ids"][:, None] == torch.arange(L, device=x.device)).float() * s["scale"]
    low = (x @ s["a"].float().reshape(L * R, -1).T).reshape(T, L, R) * mine[:, :, None]
    y = x @ s["w"].float().T + low.reshape(T, L * R) @ s["b"].float().permute(0, 2, 1).reshape(L * R, -1)
    return _act_plain(y, c["act"])


def run(state):
    s, c = state, state["case"]
    if own:
        import moe_decode_layer_logits_gb300 as M

        if c["op"] == "route":
            ids, w = M.moe_group_topk_route(s["logits"], c["k"], 2.5, bias=s["bias"], n_group=c["n_group"],
                                            topk_group=c["topk_group"], group_top=c["group_top"], scores=c["scores"],
                                            renormalize=c["renorm"])
            return dict(ids=ids, w=w)
        if c["op"] == "map":
            row_map, row_token, offsets, counts = M.moe_expert_map(s["ids"], c["E"], block=c["block"])
            return dict(row_map=row_map, row_token=row_token, offsets=offsets, counts=counts)
        act = None if c["act"] == "none" else c["act"]
        if c["op"] == "expert":
            return M.moe_expert_linear(s["x"], s["w"], s["offsets"], s["counts"], row_token=s["row_token"], act=act)
        return M.moe_adapter_linear(s["x"], s["w"], s["a"], s["b"], s["ids"], s["scale"], act=act)
    if c["op"] == "route":
        return _route_plain(c, s["logits"], s["bias"])
    if c["op"] == "map":
        return _map_plain(c, s["ids"])
    if c["op"] == "expert":
        return _expert_plain(s, c)
    return _adapter_plain(s, c)


def work(case):
    c = case
    T = c["T"]
    if c["op"] == "route":
        return dict(bytes=T * c["E"] * 4 + (c["E"] * 4 if c["bias"] else 0) + T * c["k"] * 8, flops=T * c["E"] * 8)
    if c["op"] == "map":
        return dict(bytes=T * c["k"] * 8 + _rows_needed(c) * 4 + c["E"] * 8 + 4, flops=0)
    K, N = c["K"], c["N"]
    out = N if c["act"] == "none" else N // 2
    if c["op"] == "expert":
        n = T * c["k"]
        active = c["E"] * (1 - (1 - min(1.0, c["k"] / c["E"])) ** T)  # expected, with even experts
        return dict(bytes=active * N * K * 2 + (T if c["gather"] else n) * K * 2 + (n * 4 if c["gather"] else 0)
                    + c["E"] * 8 + n * out * 2, flops=2 * n * N * K)
    used = c["L"] * (1 - (1 - 0.875 / c["L"]) ** c["requests"])  # expected adapters in use
    return dict(bytes=N * K * 2 + used * c["R"] * (K + N) * 2 + T * (K + out) * 2 + T * 4 + c["L"] * 4,
                flops=2 * T * N * K + 2 * T * c["R"] * (K + N))


# ------------------------------------------------------------------ 64-bit definition


def _silu_product(y, act):
    if act == "none":
        return y
    half = y.shape[-1] // 2
    gate, up = y[..., :half], y[..., half:]
    return gate * torch.special.expit(gate) * up


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "map":
        return None  # whole numbers throughout
    if c["op"] == "route":
        z = s["logits"].double()
        score = z.exp() / z.exp().sum(1, keepdim=True) if c["scores"] == "softmax" else 1 / (1 + (-z).exp())
        by = score if s["bias"] is None else score + s["bias"].double()
        size = c["E"] // c["n_group"]
        best = torch.stack([by[:, i * size:(i + 1) * size].topk(min(size, c["group_top"]), dim=1).values.sum(1)
                            for i in range(c["n_group"])], dim=1)
        for _ in range(c["n_group"] - c["topk_group"]):  # take the worst group out, the highest index among equals
            low = (best == best.min(1, keepdim=True).values).int()
            at = c["n_group"] - 1 - low.flip(1).argmax(1)
            best[torch.arange(len(at), device=at.device), at] = math.inf
            lanes = at[:, None] * size + torch.arange(size, device=at.device)
            by = by.scatter(1, lanes, -math.inf)
        picked = []
        for _ in range(c["k"]):
            at = by.argmax(1, keepdim=True)
            picked.append(score.gather(1, at))
            by = by.scatter(1, at, -math.inf)
        w = torch.cat(picked, 1)
        return dict(ids=None, w=2.5 * (w / w.sum(1, keepdim=True) if c["renorm"] else w))
    if c["op"] == "expert":
        n, out = c["T"] * c["k"], c["N"] if c["act"] == "none" else c["N"] // 2
        y = torch.empty(n, out, dtype=torch.float64, device=DEV)
        ends = torch.cumsum(s["counts"], 0).tolist()
        for e in range(c["E"]):
            lo, hi = (ends[e - 1] if e else 0), ends[e]
            if hi > lo:
                rows = s["x"][lo:hi] if s["row_token"] is None else s["x"][s["row_token"][lo:hi].long()]
                y[lo:hi] = _silu_product(torch.einsum("rk,nk->rn", rows.double(), s["w"][e].double()), c["act"])
        return y
    y = torch.einsum("tk,nk->tn", s["x"].double(), s["w"].double())
    for i in range(c["L"]):
        at = (s["ids"] == i).nonzero()[:, 0]
        if len(at):
            y[at] += s["scale"][i].double() * ((s["x"][at].double() @ s["a"][i].double().T) @ s["b"][i].double().T)
    return _silu_product(y, c["act"])
