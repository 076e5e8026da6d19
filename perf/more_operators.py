"""Measured cases of routing by scores and of low-rank adapters.

Three operators, each in a plain form (elementary torch operations; decisions in
fp64, sums in fp32) and, where `own` is true, as the call a user makes of the
library:

  route  experts and weights of each token from its logits: softmax or sigmoid
         scores, a bias that takes part in the choice alone, choice of groups,
         top-k, weights as they are or renormalised
  lists  the same, with the pairs grouped by expert
  lora   y[m] += scale_s B_s (A_s x_m) for the rows m of adapter s

Sizes are those of the page-shaped layer (hidden 6144, 384 experts, 8 active,
blocks of 8 drafted tokens, batches of 8, 64, 512 and 8192 tokens) and odd ones."""

import math

import torch

own = False

H, E, K8 = 6144, 384, 8
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one drafted block of 8 tokens: latency
        {"name": "route_t8", "op": "route", "T": 8, "E": E, "k": K8, "score": "sigmoid", "bias": True,
         "groups": 1, "keep": 1, "best": 2, "norm": True, "scale": 2.5},
        # 8 sequences of softmax-scored routing, weights as they are, the best expert stands for its group
        {"name": "route_soft_t64", "op": "route", "T": 64, "E": 160, "k": 6, "score": "softmax", "bias": False,
         "groups": 8, "keep": 3, "best": 1, "norm": False, "scale": 16.0},
        # sizes that are powers of nothing, groups of 29
        {"name": "route_odd", "op": "route", "T": 1021, "E": 145, "k": 5, "score": "sigmoid", "bias": True,
         "groups": 5, "keep": 2, "best": 2, "norm": True, "scale": 1.0},
        # a prefill chunk, groups and bias
        {"name": "route_t8192", "op": "route", "T": 8192, "E": E, "k": K8, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "best": 2, "norm": True, "scale": 2.5},
        # what the layer starts with at one drafted block
        {"name": "lists_t8", "op": "lists", "T": 8, "E": E, "k": K8, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "best": 2, "norm": True, "scale": 2.5},
        # and for a prefill chunk, softmax scores with a bias
        {"name": "lists_t8192", "op": "lists", "T": 8192, "E": E, "k": K8, "score": "softmax", "bias": True,
         "groups": 1, "keep": 1, "best": 1, "norm": True, "scale": 1.0},
        # one request decoding one token with its adapter: latency
        {"name": "lora_t1", "op": "lora", "M": 1, "K": 2048, "N": 2048, "r": 8, "S": 4, "per": 1, "bare": 0.0, "out": "bf16"},
        # one drafted block beside a dense projection
        {"name": "lora_t8", "op": "lora", "M": 8, "K": H, "N": 4096, "r": 16, "S": 8, "per": 8, "bare": 0.0, "out": "bf16"},
        # 64 sequences of 8 drafted tokens, each with an adapter of its own choice, beside the router's logits
        {"name": "lora_router_t512", "op": "lora", "M": 512, "K": H, "N": E, "r": 16, "S": 64, "per": 8, "bare": 0.1, "out": "f32"},
        # the same requests beside an expert-sized output projection
        {"name": "lora_t512", "op": "lora", "M": 512, "K": 2048, "N": H, "r": 32, "S": 32, "per": 8, "bare": 0.1, "out": "bf16"},
        # ragged: odd rank, columns and rows, a third of the requests without an adapter
        {"name": "lora_odd", "op": "lora", "M": 333, "K": 1352, "N": 1001, "r": 13, "S": 7, "per": 5, "bare": 0.33, "out": "f32"},
        # prefill chunks of eight requests: memory bound
        {"name": "lora_t8192", "op": "lora", "M": 8192, "K": H, "N": 4096, "r": 64, "S": 8, "per": 1024, "bare": 0.0, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "lists", "lora", "lora"])
    if op == "lora":
        m = _log_int(rng, 1, 8192)
        r = rng.choice([4, 8, 16, 16, 24, 32, 64, _log_int(rng, 1, 64)])
        return {"op": op, "M": m, "K": 8 * _log_int(rng, 1, H // 8), "N": _log_int(rng, 1, 4096), "r": r,
                "S": _log_int(rng, 1, max(1, min(64, 512 // r))), "per": _log_int(rng, 1, 1024),
                "bare": rng.choice([0.0, 0.1, 0.5]), "out": rng.choice(["f32", "bf16"]) if m <= 4096 else "bf16"}
    groups = rng.choice([1, 1, 2, 4, 5, 8, 16])
    size = _log_int(rng, 2, E // groups)
    keep = rng.randint(1, groups)
    return {"op": op, "T": _log_int(rng, 1, 8192), "E": groups * size, "k": rng.randint(1, min(8, keep * size)),
            "score": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.6, "groups": groups, "keep": keep,
            "best": rng.choice([1, 2]), "norm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5])}


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if case["op"] != "lora":
        t, e, k = case["T"], case["E"], case["k"]
        # experts of unlike popularity, which the bias evens out as a balancing step does: in steps of 1/1024
        skew = 0.7 * randn(e)
        s["logits"] = 1.5 * randn(t, e) + skew
        step = 1024.0 * (1.0 if case["score"] == "sigmoid" else e / 8)
        s["bias"] = torch.round(-60.0 * skew) / step if case["bias"] else None
        new = lambda n, d: torch.empty(n, dtype=d, device="cuda")  # noqa: E731
        s["out"] = [new((t, k), torch.int32), new((t, k), torch.float32)]
        if case["op"] == "lists":
            s["out"] += [new(n, torch.int32) for n in (e, e + 1, t * k, t * k)]
            # 4 E bytes for each 1024 pairs is enough scratch for the grouping
            s["scratch"] = new(max(4, 4 * e * (t * k // 1024 + 1)), torch.uint8)
        return s
    m, k, n, r, a = case["M"], case["K"], case["N"], case["r"], case["S"]
    requests = -(-m // case["per"])
    slot = torch.randint(0, a, (requests,), device="cuda", generator=g)
    bare = torch.rand(requests, device="cuda", generator=g) < case["bare"]
    slot = torch.where(bare, torch.full_like(slot, -1), slot).repeat_interleave(case["per"])[:m]
    s["slot"] = slot
    s["x"] = randn(m, k).bfloat16()
    s["a"] = (randn(a, r, k) / math.sqrt(k)).bfloat16()
    s["b"] = (randn(a, n, r) / math.sqrt(r)).bfloat16()
    s["scale"] = 0.25 + torch.rand(a, device="cuda", generator=g)
    s["y"] = randn(m, n).to(DTYPES[case["out"]])
    # the rows of each adapter, ascending: made once for a batch and used by all of its projections
    key = torch.where(slot < 0, torch.full_like(slot, a), slot)
    s["rows"] = torch.sort(key, stable=True).indices.int()
    s["offsets"] = torch.zeros(a + 1, dtype=torch.int32, device="cuda")
    s["offsets"][1:] = torch.bincount(key, minlength=a + 1)[:a].cumsum(0)
    return s


# ---- one pass ------------------------------------------------------------------

def _first(v, n):
    """Indices of the n largest of each row, descending, the lower index first where two are equal."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :n]


def _plain_route(s):
    l, e, k = s["logits"].double(), s["E"], s["k"]
    if s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        score = torch.exp(l - l.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    c = score if s["bias"] is None else score + s["bias"].double()
    order = l if s["bias"] is None else c
    if s["groups"] > 1:
        g = torch.sort(c.view(-1, s["groups"], e // s["groups"]), dim=2, descending=True).values[:, :, :s["best"]].sum(2)
        kept = torch.zeros_like(g, dtype=torch.bool).scatter_(1, _first(g, s["keep"]), True)
        order = torch.where(kept.repeat_interleave(e // s["groups"], 1), order, torch.full_like(order, -math.inf))
    ids = _first(order, k)
    w = score.gather(1, ids)
    if s["norm"]:
        w = w / w.sum(1, keepdim=True)
    return [ids.int(), (w * s["scale"]).float()]


def _plain_lists(ids, e):
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat, minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = counts.cumsum(0)
    pairs = torch.sort(flat, stable=True).indices
    row = torch.empty_like(pairs)
    row[pairs] = torch.arange(len(pairs), device=ids.device)
    return [v.int() for v in (counts, offsets, pairs, row)]


def _plain_lora(s):
    # the products with every adapter's A, those of other adapters than the row's own set to 0, then with every B
    a, b, slot = s["a"].float(), s["b"].float(), s["slot"]
    n_a, r, k = a.shape
    mine = torch.where(slot[:, None] == torch.arange(n_a, device=slot.device), s["scale"], torch.zeros_like(s["scale"]))
    t = (s["x"].float() @ a.view(n_a * r, k).t()).view(-1, n_a, r) * mine[:, :, None]
    y = s["y"].float() + t.view(-1, n_a * r) @ b.transpose(1, 2).reshape(n_a * r, -1)
    return s["y"].copy_(y)


def run(s):
    if own:
        import mxfp4_moe_expert_route_amd as mm
        if s["op"] == "lora":
            return mm.lora_add(s["x"], s["rows"], s["offsets"], s["a"], s["b"], s["y"], scale=s["scale"])
        rule = {"bias": s["bias"], "score": s["score"], "groups": s["groups"], "topk_groups": s["keep"],
                "group_best": s["best"], "renormalise": s["norm"], "scale": s["scale"]}
        if s["op"] == "route":
            return mm.moe_route_scored(s["logits"], s["k"], **rule, topk_ids=s["out"][0], topk_w=s["out"][1])
        ids, w, counts, offsets, pairs, row = s["out"]
        return mm.moe_route_scored_permute(s["logits"], s["k"], **rule, topk_ids=ids, topk_w=w, counts=counts,
                                           offsets=offsets, sorted_pairs=pairs, pair_to_row=row, workspace=s["scratch"])
    if s["op"] == "lora":
        return _plain_lora(s)
    out = _plain_route(s)
    return out + _plain_lists(out[0], s["E"]) if s["op"] == "lists" else out


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    if case["op"] == "lora":
        m, k, n, r = case["M"], case["K"], case["N"], case["r"]
        requests = -(-m // case["per"]) * (1.0 - case["bare"])
        used = case["S"] * (1.0 - (1.0 - 1.0 / case["S"]) ** requests) if case["S"] > 1 else min(1.0, requests)
        rows = m * (1.0 - case["bare"])
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": rows * (2.0 * k + 2.0 * n * size + 4) + 2.0 * used * r * (k + n), "flops": 2.0 * rows * r * (k + n)}
    t, e, k = case["T"], case["E"], case["k"]
    lists = 8.0 * t * k + 8.0 * e if case["op"] == "lists" else 0.0
    return {"bytes": 4.0 * t * e + (4.0 * e if case["bias"] else 0.0) + 8.0 * t * k + lists, "flops": 10.0 * t * e}


# ---- the definition, in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        y = s["y"].double()
        for i in range(case["S"]):
            rows = (s["slot"] == i).nonzero()[:, 0]
            t = torch.matmul(s["a"][i].double(), s["x"][rows].double().t())
            y[rows] += float(s["scale"][i]) * torch.matmul(s["b"][i].double(), t).t()
        return y
    l, e, n = s["logits"].double(), case["E"], case["groups"]
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    c = p if s["bias"] is None else p + s["bias"]
    number = torch.arange(e, device="cuda")
    group = number // (e // n)
    if n > 1:
        sums = torch.stack([c[:, group == i].topk(min(case["best"], e // n), 1).values.sum(1) for i in range(n)], 1)
        # a group's place: how many are before it
        before = (sums[:, :, None] < sums[:, None, :]).sum(2)
        c = c.masked_fill((before >= case["keep"])[:, group], -math.inf)
    ids = []
    for _ in range(case["k"]):
        at = torch.where(c == c.amax(1, keepdim=True), number, e).amin(1, keepdim=True)
        ids.append(at)
        c = c.scatter(1, at, -math.inf)
    ids = torch.cat(ids, 1)
    w = p.gather(1, ids)
    w = case["scale"] * (w / w.sum(1, keepdim=True) if case["norm"] else w)
    if case["op"] == "route":
        return [ids.int(), w]
    flat = ids.flatten()
    counts = (flat[:, None] == number).sum(0) if len(flat) * e < 1 << 26 else torch.histc(flat.double(), e, 0, e)
    key = flat * len(flat) + torch.arange(len(flat), device="cuda")
    pairs = key.argsort()
    return [ids.int(), w, counts.int(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int(), pairs.int(), pairs.argsort().int()]
