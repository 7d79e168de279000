"""Timed cases of the router and of the low-rank adapters.

Three operators, each in two forms: ``own = False`` computes the plain form
(elementary torch operations in 32 bits, in 64 for the scores that a choice of
experts compares, rounded once at the end), ``own = True`` makes the calls a
user makes of the library.

logits    router logits x W^T of bf16 activations, W in bf16 or fp32, FP32 result
route     the choice of experts from the logits: softmax or sigmoid scores, a
          bias for balance, groups, top-k, renormalised and scaled weights
adapter   low-rank adapters of many requests beside a projection that they share:
          y[p] = base[p] + scale * B (A x[p]), each row with the adapter of its
          request, for one projection or for every expert's
"""
import torch

own = False
DEV = "cuda"


# --------------------------------------------------------------------- cases

def listed():
    """The timed cases (hidden size 7168, 384 experts, top-8, intermediate size
    2048: the shapes of ``workloads``; other sizes are generic)."""
    return [
        # decode of one request: latency is all that counts
        {"name": "logits_T1", "op": "logits", "T": 1, "E": 384, "H": 7168, "w": "bf16"},
        # a decode batch with a router kept in fp32
        {"name": "logits_T48_f32", "op": "logits", "T": 48, "E": 384, "H": 7168, "w": "f32"},
        # odd sizes: tokens, experts and K that fill no tile
        {"name": "logits_ragged", "op": "logits", "T": 1003, "E": 161, "H": 2088, "w": "bf16"},
        # prefill
        {"name": "logits_T8192", "op": "logits", "T": 8192, "E": 384, "H": 7168, "w": "bf16"},
        # decode of one request
        {"name": "route_T1", "op": "route", "T": 1, "E": 384, "topk": 8, "dtype": "f32", "score": "sigmoid", "bias": True,
         "groups": 1, "topk_groups": 1, "best": 1, "renorm": True, "scale": 2.5, "first": 0, "local": 384, "masked": False},
        # prefill of 16384 tokens on an expert-parallel share: seven of eight choices live elsewhere
        {"name": "route_T16384", "op": "route", "T": 16384, "E": 384, "topk": 8, "dtype": "f32", "score": "sigmoid",
         "bias": True, "groups": 1, "topk_groups": 1, "best": 1, "renorm": True, "scale": 2.5, "first": 48, "local": 48,
         "masked": False},
        # choice limited to four of eight groups, a few experts switched off, padding tokens without any expert
        {"name": "route_groups", "op": "route", "T": 4096, "E": 256, "topk": 8, "dtype": "f32", "score": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "best": 2, "renorm": True, "scale": 2.5, "first": 0, "local": 256,
         "masked": True},
        # an odd number of bf16 rows, softmax over few experts: many equal logits
        {"name": "route_softmax_bf16", "op": "route", "T": 1003, "E": 61, "topk": 6, "dtype": "bf16", "score": "softmax",
         "bias": False, "groups": 1, "topk_groups": 1, "best": 1, "renorm": False, "scale": 1.0, "first": 0, "local": 61,
         "masked": False},
        # decode of one request with its adapter, one projection
        {"name": "adapter_T1", "op": "adapter", "T": 1, "topk": 1, "E": 1, "Eg": 1, "S": 8, "rank": 16, "parts": 1,
         "K": 7168, "N": 4096, "div": 1, "out": "bf16", "none": 0.0, "runs": 1},
        # a decode batch of many requests on the gate_up weights of every expert of a small share
        {"name": "adapter_decode_experts", "op": "adapter", "T": 32, "topk": 8, "E": 8, "Eg": 64, "S": 16, "rank": 16,
         "parts": 2, "K": 7168, "N": 4096, "div": 8, "out": "bf16", "none": 0.2, "runs": 1},
        # prefill of eight requests in one chunk, one projection; one request in eight has no adapter
        {"name": "adapter_prefill_dense", "op": "adapter", "T": 4096, "topk": 1, "E": 1, "Eg": 1, "S": 8, "rank": 64,
         "parts": 1, "K": 7168, "N": 4096, "div": 1, "out": "bf16", "none": 0.125, "runs": 512},
        # prefill, down projection of every expert: one activation row per pair, FP32 sums
        {"name": "adapter_prefill_down", "op": "adapter", "T": 1024, "topk": 8, "E": 48, "Eg": 48, "S": 4, "rank": 16,
         "parts": 1, "K": 2048, "N": 7168, "div": 1, "out": "f32", "none": 0.125, "runs": 256},
    ]


def _log(rng, lo, hi):
    return lo * (hi / lo) ** rng.random()


def draw(rng):
    op = rng.choice(["logits", "route", "adapter"])
    if op == "logits":
        T = max(1, round(_log(rng, 1, 8192)))
        E = max(2, round(_log(rng, 2, 512)))
        H = 8 * max(1, round(_log(rng, 8, 896)))
        w = rng.choice(["bf16", "bf16", "f32"])
        while T * E * H * (3 if w == "f32" else 1) > 8192 * 384 * 7168:
            T //= 2
        return {"op": "logits", "T": T, "E": E, "H": H, "w": w}
    if op == "route":
        T = max(1, round(_log(rng, 1, 16384)))
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        size = max(2, round(_log(rng, 2, 512 // groups)))
        E = groups * size
        while T * E > 16384 * 384:
            T //= 2
        topk_groups = rng.randint(1, groups)
        topk = rng.randint(1, min(topk_groups * size, 16))
        local = E if rng.random() < 0.6 else max(1, E // rng.choice([2, 4, 8]))
        return {"op": "route", "T": T, "E": E, "topk": topk, "dtype": rng.choice(["f32", "f32", "bf16"]),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "topk_groups": topk_groups, "best": rng.choice([1, 2]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "first": rng.randint(0, E - local), "local": local,
                "masked": rng.random() < 0.3}
    T = max(1, round(_log(rng, 1, 4096)))
    topk = rng.choice([1, 1, 2, 4, 8])
    Eg = 1 if topk == 1 and rng.random() < 0.7 else max(topk, round(_log(rng, 2, 48)))
    E = Eg if rng.random() < 0.7 else max(1, Eg // 2)
    S = max(1, round(_log(rng, 1, 16)))
    rank = rng.choice([8, 16, 16, 24, 32, 64])
    parts = rng.choice([1, 1, 2])
    K = 8 * max(1, round(_log(rng, 8, 896)))
    N = 8 * parts * max(1, round(_log(rng, 8, 896) / parts))
    while T * topk * (K + N) > 8192 * (2048 + 7168):
        T //= 2
    while S * E * rank * (parts * K + N) > 300_000_000:
        S = max(1, S // 2)
        E = Eg = max(topk if topk > 1 else 1, Eg // 2)
    return {"op": "adapter", "T": T, "topk": topk, "E": E, "Eg": Eg, "S": S, "rank": rank, "parts": parts, "K": K, "N": N,
            "div": rng.choice([1, topk]), "out": rng.choice(["bf16", "f32"]), "none": rng.choice([0.0, 0.2]),
            "runs": rng.choice([1, 1, 64, 512])}


def work(case):
    """Bytes every input read once and every output written once; the adapters
    that a token is expected to choose count."""
    if case["op"] == "logits":
        T, E, H = case["T"], case["E"], case["H"]
        return {"bytes": T * H * 2 + E * H * (2 if case["w"] == "bf16" else 4) + T * E * 4, "flops": 2 * T * E * H}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        return {"bytes": T * E * (4 if case["dtype"] == "f32" else 2) + T * case["topk"] * 8 + (E * 4 if case["bias"] else 0),
                "flops": 8 * T * E}
    T, k, E, Eg, S, K, N, r = (case[n] for n in ("T", "topk", "E", "Eg", "S", "K", "N", "rank"))
    rows, has = T * k * E / Eg, 1.0 - case["none"]
    # requests draw their adapter at random, their tokens' experts are independent
    requests = max(1, T // case["runs"]) * has
    adapters = S * (1.0 - (1.0 - 1.0 / S) ** requests)
    slots = adapters * E * (1.0 - (1.0 - k / Eg) ** (T * has / adapters)) if Eg > 1 else adapters
    x_rows = T if case["div"] == k else T * k * E / Eg
    esize = 2 if case["out"] == "bf16" else 4
    return {"bytes": slots * r * (case["parts"] * K + N) * 2 + x_rows * has * K * 2 + rows * N * 2 * esize,
            "flops": 2 * rows * has * r * (case["parts"] * K + N)}


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _data(case, seed):
    """The plain inputs of a case."""
    g = _gen(seed)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    d = {}
    if case["op"] == "logits":
        T, E, H = case["T"], case["E"], case["H"]
        d["x"] = randn(T, H).to(torch.bfloat16)
        W = randn(E, H) * H ** -0.5
        d["W"] = W.to(torch.bfloat16) if case["w"] == "bf16" else W
    elif case["op"] == "route":
        T, E = case["T"], case["E"]
        l = randn(T, E) * 1.5 + randn(1, E) * 0.5
        if case["masked"]:
            # experts that are switched off, and padding tokens that may go nowhere
            off = rand(1, E) < 0.03
            pad = rand(T, 1) < 0.02
            l = torch.where(off | pad, torch.full_like(l, float("-inf")), l)
        d["l"] = l.to(torch.bfloat16) if case["dtype"] == "bf16" else l
        d["b"] = randn(E) * 0.05 if case["bias"] else None
    else:
        T, k, E, Eg, S, K, N, r = (case[n] for n in ("T", "topk", "E", "Eg", "S", "K", "N", "rank"))
        # every `runs` tokens are one request with one adapter, or none (-1)
        n = -(-T // case["runs"])
        a = torch.randint(0, S, (n,), generator=g, device=DEV, dtype=torch.int32)
        a = torch.where(rand(n) < case["none"], torch.full_like(a, -1), a)
        d["a"] = a.repeat_interleave(case["runs"])[:T].contiguous()
        if Eg > 1:
            ids = torch.argsort(rand(T, Eg), dim=1)[:, :k].to(torch.int32)
            d["ids"] = torch.where(ids < E, ids, torch.full_like(ids, -1)).contiguous()
        else:
            d["ids"] = None
        d["x"] = randn(T * k // case["div"], K).to(torch.bfloat16)
        lead = (S, E) if Eg > 1 else (S,)
        d["A"] = (randn(*lead, case["parts"] * r, K) * K ** -0.5).to(torch.bfloat16)
        d["B"] = (randn(*lead, N, r) * 0.3 * r ** -0.5).to(torch.bfloat16)
        d["scale"] = 0.5 + rand(S)
        d["base"] = randn(T * k, N).to(torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    return d


def _slots(case, a, ids):
    """(slot of each pair, whether the pair is on this GPU): slot = adapter * E + expert, -1 without an adapter."""
    per = a.long().repeat_interleave(case["topk"])
    e = ids.reshape(-1).long() if ids is not None else torch.zeros_like(per)
    here = e >= 0
    return torch.where((per >= 0) & here, per * case["E"] + e, torch.full_like(per, -1)), here


def prepare(case, seed):
    s = {"case": case}
    s.update(_data(case, seed))
    if not own:
        if case["op"] == "adapter":
            slot, here = _slots(case, s["a"], s["ids"])
            # rows of each slot, as a plain program groups its batch
            s["rows"] = [(int(v), torch.nonzero(slot == v).reshape(-1)) for v in torch.unique(slot).tolist() if v >= 0]
            s["here"] = None if bool(here.all()) else torch.nonzero(here).reshape(-1)
        return s
    import w4a16_int4_mixture_moe_gb300 as chord
    s["chord"] = chord
    if case["op"] == "logits":
        T, E, H = case["T"], case["E"], case["H"]
        if case["w"] == "f32":
            parts = torch.empty((3, E, H), dtype=torch.bfloat16, device=DEV)
            chord.chord_router_split_weights(s["W"], parts)
            s["W"] = parts
        s["out"] = torch.empty((T, E), dtype=torch.float32, device=DEV)
    elif case["op"] == "route":
        T, k = case["T"], case["topk"]
        s["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        s["w"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
        s["score"] = chord.SCORE_SIGMOID if case["score"] == "sigmoid" else chord.SCORE_SOFTMAX
    else:
        s["y"] = torch.zeros_like(s["base"])
        s["ws"] = torch.empty(chord.chord_adapter_workspace_bytes(case["T"], case["topk"], case["S"], case["E"], case["rank"],
                                                                  case["parts"]), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms

def _plain_logits(s):
    return s["x"].float() @ s["W"].float().t()


def _plain_scores(l, open_, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - torch.where(open_.any(dim=1, keepdim=True), top, torch.zeros_like(top)))
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total))


def _plain_route(s):
    """An expert whose logit is -inf is not available; a token with fewer
    available experts than top-k ends in id -1 and weight 0."""
    case = s["case"]
    T, E, G, k = case["T"], case["E"], case["groups"], case["topk"]
    ninf = float("-inf")
    l = s["l"].float()
    open_ = l > ninf
    # scores of the choice in 64 bits: two experts of a token may differ in the last bits only
    ld = l.double()
    p, q = (_plain_scores(v, open_, case["score"]) for v in (ld, l))
    z = p if s["b"] is None else p + s["b"].double()
    if s["b"] is None and case["best"] == 1:
        z = ld                                   # the same order, without the scores' rounding
    z = torch.where(open_, z, torch.full_like(z, ninf))
    if G > 1:
        top = torch.sort(z.reshape(T, G, E // G), dim=2, descending=True).values[:, :, :case["best"]]
        any_ = top[:, :, 0] > ninf
        gz = torch.where(top > ninf, top, torch.zeros_like(top)).sum(dim=2)
        gz = torch.where(any_, gz, torch.full_like(gz, ninf))
        order = torch.sort(gz, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, order, True)
        z = torch.where(keep.repeat_interleave(E // G, dim=1), z, torch.full_like(z, ninf))
    if s["b"] is None:
        z = torch.where(z > ninf, ld, z)         # inside the groups the logits' order is the scores'
    zs, idx = torch.sort(z, dim=1, descending=True, stable=True)
    zs, idx = zs[:, :k], idx[:, :k]
    got = zs > ninf
    w = torch.where(got, q.gather(1, idx), torch.zeros_like(q[:, :1]))
    if case["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    w = w * case["scale"]
    local = got & (idx >= case["first"]) & (idx < case["first"] + case["local"])
    return torch.where(local, idx - case["first"], torch.full_like(idx, -1)).to(torch.int32), w


def _plain_adapter(s):
    case = s["case"]
    r, parts, N = case["rank"], case["parts"], case["N"]
    A = s["A"].reshape(-1, parts * r, case["K"])
    B = s["B"].reshape(-1, N, r)
    if s["here"] is None:
        y = s["base"].clone()
    else:
        y = torch.zeros_like(s["base"])
        y[s["here"]] = s["base"][s["here"]]
    for slot, rows in s["rows"]:
        v = s["x"][rows // case["div"]].float() @ A[slot].float().t()
        b = B[slot].float()
        d = torch.cat([v[:, i * r:(i + 1) * r] @ b[i * (N // parts):(i + 1) * (N // parts)].t() for i in range(parts)], dim=1)
        y[rows] = (s["base"][rows].float() + s["scale"][slot // case["E"]] * d).to(y.dtype)
    return y


# ----------------------------------------------------------------------- run

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"logits": _plain_logits, "route": _plain_route, "adapter": _plain_adapter}[op](s)
    chord = s["chord"]
    if op == "logits":
        chord.chord_router_logits(s["x"], s["W"], s["out"])
        return s["out"]
    if op == "route":
        chord.chord_moe_route(s["l"], s["ids"], s["w"], score=s["score"], bias=s["b"], groups=case["groups"],
                              topk_groups=case["topk_groups"], group_best=case["best"], renormalize=case["renorm"],
                              scale=case["scale"], first=case["first"], E_local=case["local"])
        return s["ids"], s["w"]
    chord.chord_adapter_add(s["x"], case["div"], s["a"], s["ids"], s["A"], s["B"], s["scale"], s["base"], s["y"], s["ws"])
    return s["y"]


# --------------------------------------------------------------------- exact

def _exact_route(case, d):
    """One choice after the other, on scores in 64 bits."""
    T, E, G = case["T"], case["E"], case["groups"]
    v = d["l"].double()
    alive = ~torch.isinf(v)
    low = torch.full_like(v, -float("inf"))
    if case["score"] == "sigmoid":
        p = torch.special.expit(v)
    else:
        p = torch.where(alive, torch.special.softmax(torch.where(alive.any(1, keepdim=True), v, torch.zeros_like(v)), dim=1),
                        torch.zeros_like(v))
    rank = v.clone() if d["b"] is None else p + d["b"].double()
    rank = torch.where(alive, rank, low)
    if G > 1:
        by = rank if d["b"] is not None or case["best"] == 1 else torch.where(alive, p, low)
        by = by.reshape(T, G, E // G)
        first, at = by.max(dim=2)
        score = first
        if case["best"] == 2 and E // G > 1:
            rest = by.scatter(2, at.unsqueeze(2), -float("inf")).max(dim=2).values
            score = torch.where(torch.isinf(rest), first, first + rest)
        chosen = torch.zeros((T, G), dtype=torch.bool, device=v.device)
        g = torch.arange(G, device=v.device).expand(T, G)
        for _ in range(case["topk_groups"]):
            left = torch.where(chosen, torch.full_like(score, -float("inf")), score)
            best = left.max(dim=1, keepdim=True).values
            at = torch.where((left == best) & ~chosen, g, torch.full_like(g, G)).min(dim=1, keepdim=True).values
            chosen.scatter_(1, at, True)
        rank = torch.where(chosen.repeat_interleave(E // G, dim=1), rank, low)
    ids, ws = [], []
    col = torch.arange(E, device=v.device).expand(T, E)
    for _ in range(case["topk"]):
        best = rank.max(dim=1, keepdim=True).values
        have = ~torch.isinf(best)
        at = torch.where((rank == best) & have, col, torch.full_like(col, E)).min(dim=1, keepdim=True).values
        safe = at.clamp(max=E - 1)
        ws.append(torch.where(have, p.gather(1, safe), torch.zeros_like(best)))
        ids.append(torch.where(have, at, torch.full_like(at, -1)))
        rank = torch.where(have & (col == at), low, rank)
    ids, w = torch.cat(ids, 1), torch.cat(ws, 1)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    ids = ids - case["first"]
    ids = torch.where((ids >= 0) & (ids < case["local"]), ids, torch.full_like(ids, -1))
    return ids.to(torch.int32), w * case["scale"]


def exact(case, seed):
    d = _data(case, seed)
    if case["op"] == "logits":
        W = d["W"].double().t().contiguous()
        return torch.cat([c.double() @ W for c in d["x"].split(1024)])
    if case["op"] == "route":
        return _exact_route(case, d)
    parts, r, N, k = case["parts"], case["rank"], case["N"], case["topk"]
    y = torch.zeros(d["base"].shape, dtype=torch.float64, device=DEV)
    S, E = case["S"], case["E"]
    A = d["A"].view(S, E, parts, r, case["K"])
    B = d["B"].view(S, E, parts, N // parts, r)
    pair = torch.arange(case["T"] * k, device=DEV)
    expert = torch.zeros_like(pair) if d["ids"] is None else d["ids"].flatten().long()
    adapter = d["a"].long()[torch.div(pair, k, rounding_mode="floor")]
    bare = pair[(expert >= 0) & (adapter < 0)]
    y[bare] = d["base"][bare].double()
    for a in range(S):
        for e in range(E):
            mine = pair[(adapter == a) & (expert == e)]
            if mine.numel() == 0:
                continue
            x = d["x"][torch.div(mine, case["div"], rounding_mode="floor")].double()
            delta = [(x @ A[a, e, i].double().t()) @ B[a, e, i].double().t() for i in range(parts)]
            y[mine] = d["base"][mine].double() + d["scale"][a].double() * torch.cat(delta, dim=1)
    return y
