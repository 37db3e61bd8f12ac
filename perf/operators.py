"""Operators around the compressed matmuls of a language model's feed-forward
part, as a serving step uses them, each in its plain form (elementary torch
operations) and as the calls of this library:

  route     routing of tokens to experts: scores, selection, weights, and the
            expert order of the routed rows
  gate_up   the routed experts' gate and up products with the gated activation
  down      the routed experts' down product, joined per token with the weights
  lora      low-rank adapters of many requests beside a shared projection

`own` selects which of the two `run` computes.
"""
import math

import torch

own = False

DEV = "cuda"
FLT_MAX = torch.finfo(torch.float32).max


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 8 sequences, many small experts, plain softmax gate
        {"name": "route decode", "op": "route", "t": 8, "e": 128, "top_k": 8, "dtype": "bf16", "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_score": "max", "renorm": True, "scale": 1.0, "padded": False},
        # a prefill chunk under a balanced, group-limited sigmoid gate
        {"name": "route grouped prefill", "op": "route", "t": 8192, "e": 256, "top_k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_score": "top2", "renorm": True,
         "scale": 2.5, "padded": False},
        # a ragged batch padded to its longest sequence: the padding rows route nowhere
        {"name": "route padded odd", "op": "route", "t": 1537, "e": 60, "top_k": 4, "dtype": "f32", "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_score": "max", "renorm": False, "scale": 1.0, "padded": True},
        # one sequence's next token through its 8 experts: a latency-bound stream of their weights
        {"name": "gate_up one token", "op": "gate_up", "t": 1, "e": 128, "n": 768, "k": 2048, "top_k": 8},
        # a decode batch: most experts are read, each for a few tokens
        {"name": "gate_up decode batch", "op": "gate_up", "t": 64, "e": 128, "n": 768, "k": 2048, "top_k": 8},
        # a prefill chunk: tensor-core work, ragged over the experts
        {"name": "gate_up prefill", "op": "gate_up", "t": 4096, "e": 128, "n": 768, "k": 2048, "top_k": 8},
        {"name": "down decode", "op": "down", "t": 16, "e": 128, "n": 2048, "k": 768, "top_k": 8},
        # an odd number of tokens over fewer, larger experts
        {"name": "down prefill odd", "op": "down", "t": 2331, "e": 16, "n": 4096, "k": 1408, "top_k": 2},
        # decode: every sequence has an adapter of its own or none
        {"name": "lora decode", "op": "lora", "t": 32, "n": 4096, "k": 4096, "adapters": 48, "max_rank": 16,
         "runs": False},
        # one sequence, the largest projection
        {"name": "lora one token", "op": "lora", "t": 1, "n": 14336, "k": 4096, "adapters": 8, "max_rank": 64,
         "runs": True},
        # a prefill batch: long runs of rows with one adapter each
        {"name": "lora prefill", "op": "lora", "t": 4096, "n": 14336, "k": 4096, "adapters": 8, "max_rank": 32,
         "runs": True},
        # a mixed batch of ragged prompts and single tokens
        {"name": "lora mixed odd", "op": "lora", "t": 777, "n": 4096, "k": 14336, "adapters": 20, "max_rank": 64,
         "runs": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "gate_up", "down", "lora"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        e = groups * rng.randint(max(2, 8 // groups), 256 // groups)
        top_groups = rng.randint(1, groups)
        return {"op": op, "t": _log(rng, 1, 8192), "e": e, "top_k": rng.randint(1, min(10, e // groups * top_groups)),
                "dtype": rng.choice(["f32", "bf16"]), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups,
                "group_score": rng.choice(["max", "top2"]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 1.5, 2.5]), "padded": rng.random() < 0.3}
    if op == "lora":
        return {"op": op, "t": _log(rng, 1, 4096), "n": 64 * rng.randint(8, 224), "k": 64 * rng.randint(8, 224),
                "adapters": _log(rng, 1, 64), "max_rank": rng.choice([8, 16, 24, 32, 64]), "runs": rng.random() < 0.6}
    while True:
        e = _log(rng, 4, 128)
        c = {"op": op, "t": _log(rng, 1, 4096), "e": e, "n": 64 * rng.randint(4, 64), "k": 64 * rng.randint(4, 64),
             "top_k": rng.randint(1, min(8, e))}
        if c["t"] * c["e"] * c["n"] * c["k"] <= 4096 * 128 * 768 * 2048 and c["e"] * c["n"] * c["k"] <= 128 * 768 * 2048:
            return c


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(torch.bfloat16)


def _order_of(ids, groups):
    """Rows in group order (stable; rows of no group last), the groups' offsets, and each row's place."""
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, groups, flat).long()
    order = torch.sort(key, stable=True).indices
    offsets = torch.zeros(groups + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(torch.bincount(key, minlength=groups + 1)[:groups], 0)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device=DEV)
    slot = torch.where(flat < 0, -1, slot).reshape(ids.shape)
    return order.int(), offsets.int(), slot.int()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    t = case["t"]
    if case["op"] == "route":
        e = case["e"]
        # gate outputs of a trained router: spread over tokens, some experts more popular than others
        logits = torch.randn(t, e, device=DEV, generator=g) * 1.5 + torch.randn(e, device=DEV, generator=g) * 0.5
        if case["padded"]:
            lengths = torch.rand(t, 1, device=DEV, generator=g)
            logits = torch.where(lengths < 0.25, float("-inf"), logits)
        s["logits"] = logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits
        s["bias_t"] = torch.randn(e, device=DEV, generator=g) * 0.02 if case["bias"] else None
        return s
    if case["op"] == "lora":
        n, k, a, r = case["n"], case["k"], case["adapters"], case["max_rank"]
        s["x"] = _normal(g, t, k)
        s["a"] = _normal(g, a, r, k, std=1.0 / math.sqrt(k))
        s["b"] = _normal(g, a, n, r, std=0.1)
        s["base"] = torch.randn(t, n, device=DEV, generator=g)
        # adapters' own ranks up to the slots' width, whole slots most often
        s["ranks"] = torch.where(torch.rand(a, device=DEV, generator=g) < 0.5, r,
                                 torch.randint(1, r + 1, (a,), device=DEV, generator=g)).int()
        s["scales"] = torch.rand(a, device=DEV, generator=g) * 1.5 + 0.5
        if case["runs"]:   # requests of several rows each: about as many requests as adapters
            cuts = (torch.rand(t, device=DEV, generator=g) < min(1.0, (a + 1) / t)).long()
            of_request = torch.randint(-1, a, (t + 1,), device=DEV, generator=g)
            s["ids"] = of_request[torch.cumsum(cuts, 0)].int()
        else:
            s["ids"] = torch.randint(-1, a, (t,), device=DEV, generator=g).int()
        if t == 1:
            s["ids"] = torch.randint(0, a, (1,), device=DEV, generator=g).int()
        s["out"] = torch.empty(t, n, dtype=torch.float32, device=DEV)
        return s
    e, n, k, top = case["e"], case["n"], case["k"], case["top_k"]
    # distinct experts for each token, some more popular than others
    gate = torch.randn(t, e, device=DEV, generator=g) + torch.randn(e, device=DEV, generator=g) * 0.5
    s["ids"] = torch.topk(gate, top, dim=1).indices.int()
    s["order"], s["offsets"], s["slot"] = _order_of(s["ids"], e)
    if case["op"] == "gate_up":
        s["x"] = _normal(g, t, k)
        s["w"] = _normal(g, e, 2 * n, k, std=0.02)   # each expert's gate rows, then its up rows
        s["out"] = torch.empty(t * top, n, dtype=torch.bfloat16, device=DEV)
    else:
        s["x"] = _normal(g, t * top, k, std=0.5)     # the activations, in expert order
        s["w"] = _normal(g, e, n, k, std=0.02)
        p = torch.rand(t, top, device=DEV, generator=g) + 0.1
        s["weights"] = p / p.sum(1, keepdim=True)
        s["out"] = torch.empty(t, n, dtype=torch.float32, device=DEV)
    return s


# --------------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _own(state)
    return {"route": _route, "gate_up": _gate_up, "down": _down, "lora": _lora}[state["op"]](state)


def _own(s):
    from decode_gemm_exponent_b200 import uw
    if s["op"] == "route":
        r = uw.route_experts(s["logits"], s["top_k"], score=s["score"], bias=s["bias_t"], n_groups=s["groups"],
                             top_groups=s["top_groups"], group_score=s["group_score"], renormalize=s["renorm"],
                             scale=s["scale"], out=s.get("routing"))
        s["routing"] = r      # a serving loop keeps its buffers
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "order": r.order, "slot": r.slot}
    if s["op"] == "lora":
        ws = s.get("ws")
        if ws is None:
            ws = s["ws"] = uw.new_workspace(uw.lora_workspace_size(s["t"], s["k"], s["n"], s["adapters"], s["max_rank"]), DEV)
        return uw.lora_add(s["x"], s["a"], s["b"], s["ids"], s["base"], ranks=s["ranks"], scales=s["scales"], out=s["out"],
                           ws=ws)
    routing = uw.Routing(s["ids"], s.get("weights"), s["offsets"], s["order"], s["slot"])
    if s["op"] == "gate_up":
        n = s["n"]
        return uw.expert_gate_up(s["x"], s["w"][:, :n], s["w"][:, n:], routing, out=s["out"])
    rows = s.get("rows")
    if rows is None:
        rows = s["rows"] = torch.empty(s["x"].shape[0], s["n"], dtype=torch.float32, device=DEV)
    uw.expert_matmul(s["x"], s["w"], routing, out=rows)
    return uw.expert_combine(rows, routing, out=s["out"])


def _route(s):
    e, top, groups = s["e"], s["top_k"], s["groups"]
    # 64 bits: which of two scores next to each other is larger decides an index
    l = s["logits"].double()
    dead = torch.isnan(l) | (l == -math.inf)
    l = torch.clamp(torch.where(dead, 0.0, l), max=FLT_MAX)
    if s["score"] == "softmax":
        m = torch.where(dead, -math.inf, l).amax(1, keepdim=True)
        p = torch.where(dead, 0.0, torch.exp(l - torch.where(m == -math.inf, 0.0, m)))
        score = p / torch.clamp(p.sum(1, keepdim=True), min=1e-300)
    else:
        score = torch.where(dead, 0.0, 1.0 / (1.0 + torch.exp(-l)))
    # without a bias the order of the scores is the order of the logits
    choice = torch.where(dead, -math.inf, l if s["bias_t"] is None else score + s["bias_t"].double())
    if groups > 1:
        per = choice.reshape(-1, groups, e // groups)
        if s["group_score"] == "max":
            value = per.amax(2)
        else:
            by = torch.where(dead, -math.inf, score + (0.0 if s["bias_t"] is None else s["bias_t"].double()))
            best = torch.sort(by.reshape(-1, groups, e // groups), dim=2, descending=True).values[:, :, :2]
            value = best[:, :, 0] + torch.where(best[:, :, -1] == -math.inf, 0.0, best[:, :, -1]) * (e // groups > 1)
        kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(keep[:, :, None], per, -math.inf).reshape(-1, e)
    best = torch.sort(choice, dim=1, descending=True, stable=True)
    ids = best.indices[:, :top]
    none = best.values[:, :top] == -math.inf
    w = torch.where(none, 0.0, torch.gather(score, 1, ids))
    if s["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    ids = torch.where(none, -1, ids).int()
    order, offsets, slot = _order_of(ids, e)
    return {"ids": ids, "weights": (w * s["scale"]).float(), "offsets": offsets, "order": order, "slot": slot}


def _gate_up(s):
    e, n, k, top = s["e"], s["n"], s["k"], s["top_k"]
    # every expert on every token, then the routed rows
    y = (s["x"].float() @ s["w"].float().reshape(e * 2 * n, k).T).reshape(-1, e, 2 * n)
    j = s["order"].long()
    y = y[j // top, s["ids"].reshape(-1)[j].long()]
    gate, up = y[:, :n], y[:, n:]
    return (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)


def _down(s):
    e, top, t = s["e"], s["top_k"], s["t"]
    j = s["order"].long()
    expert = s["ids"].reshape(-1)[j].long()
    padded = torch.zeros(e, t, s["k"], device=DEV)
    padded[expert, j // top] = s["x"].float()
    y = padded @ s["w"].float().transpose(1, 2)
    rows = y[s["ids"].long(), torch.arange(t, device=DEV)[:, None]]
    return (rows * s["weights"][:, :, None]).sum(1)


def _lora(s):
    a, r, n = s["adapters"], s["max_rank"], s["n"]
    v = (s["x"].float() @ s["a"].float().reshape(a * r, -1).T).reshape(-1, a, r)
    mine = s["ids"][:, None] == torch.arange(a, device=DEV)
    used = torch.arange(r, device=DEV) < s["ranks"][:, None]
    v = torch.where(mine[:, :, None] & used, v * s["scales"][:, None], 0.0)
    return s["base"] + v.reshape(-1, a * r) @ s["b"].float().transpose(1, 2).reshape(a * r, n)


# --------------------------------------------------------------------------- what a pass cannot do without

def _routed(t, e, top):
    """Experts that t tokens reach, about, with `top` distinct ones each."""
    return e * (1.0 - (1.0 - top / e) ** t)


def work(case):
    t = case["t"]
    if case["op"] == "route":
        size = 2 if case["dtype"] == "bf16" else 4
        slots = t * case["top_k"]
        return {"bytes": t * case["e"] * size + slots * 16 + 4 * (case["e"] + 1) + (4 * case["e"] if case["bias"] else 0),
                "flops": 8 * t * case["e"]}
    n, k = case["n"], case["k"]
    if case["op"] == "lora":
        a, r = case["adapters"], case["max_rank"]
        used = a * (1.0 - (1.0 - 1.0 / (a + 1)) ** t)
        return {"bytes": 2 * t * k + 8 * t * n + 0.75 * used * r * 2 * (n + k), "flops": 2 * 0.75 * t * r * (n + k)}
    rows, used = t * case["top_k"], _routed(t, case["e"], case["top_k"])
    if case["op"] == "gate_up":
        return {"bytes": 2 * t * k + used * 2 * n * k * 2 + rows * n * 2, "flops": 2.0 * rows * 2 * n * k}
    return {"bytes": 2 * rows * k + used * n * k * 2 + 4 * t * n, "flops": 2.0 * rows * n * k + 2.0 * rows * n}


# --------------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "gate_up": _exact_gate_up, "down": _exact_down, "lora": _exact_lora}[case["op"]](s)


def _exact_route(s):
    e, top, groups = s["e"], s["top_k"], s["groups"]
    l = s["logits"].double()
    alive = l > -math.inf                       # false for NaN too
    l = torch.where(alive, l.clamp(max=FLT_MAX), -math.inf)
    if s["score"] == "softmax":
        score = torch.nan_to_num(torch.softmax(l, 1))
    else:
        score = torch.sigmoid(l)
    bias = torch.zeros(e, dtype=torch.float64, device=DEV) if s["bias_t"] is None else s["bias_t"].double()
    value = torch.where(alive, score + bias, -math.inf)
    pick = l.clone() if s["bias_t"] is None else value.clone()
    if groups > 1:
        v = (pick if s["group_score"] == "max" else value).reshape(-1, groups, e // groups).clone()
        first = v.max(2)
        total = first.values.clone()
        if s["group_score"] == "top2" and e // groups > 1:
            v.scatter_(2, first.indices[:, :, None], -math.inf)
            second = v.max(2).values
            total = total + torch.where(second > -math.inf, second, torch.zeros_like(second))
        keep = torch.zeros_like(total, dtype=torch.bool)
        place = torch.arange(groups, device=DEV)
        for _ in range(s["top_groups"]):
            left = torch.where(keep, -math.inf, total)
            hit = (left == left.amax(1, keepdim=True)) & ~keep
            at = torch.where(hit, place, groups).amin(1, keepdim=True)
            keep |= place == at
        pick = torch.where(keep.repeat_interleave(e // groups, 1), pick, -math.inf)
    place = torch.arange(e, device=DEV)
    ids, w = [], []
    for _ in range(top):
        hit = (pick == pick.amax(1, keepdim=True)) & (pick > -math.inf)
        at = torch.where(hit, place, e).amin(1)
        found = at < e
        at = torch.where(found, at, 0)
        ids.append(torch.where(found, at, -1))
        w.append(torch.where(found, score.gather(1, at[:, None])[:, 0], 0.0))
        pick = torch.where((place == at[:, None]) & found[:, None], -math.inf, pick)
    ids, w = torch.stack(ids, 1), torch.stack(w, 1)
    if s["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    # the order holds by the equality of whole numbers with the plain form alone
    return {"ids": ids.int(), "weights": w * s["scale"], "offsets": None, "order": None, "slot": None}


def _exact_gate_up(s):
    n, top = s["n"], s["top_k"]
    out = torch.empty(s["t"] * top, n, dtype=torch.float64, device=DEV)
    at = s["offsets"].tolist()
    token = s["order"].long() // top
    for i in range(s["e"]):
        rows = s["x"][token[at[i]:at[i + 1]]].double()
        gate = rows @ s["w"][i, :n].double().T
        out[at[i]:at[i + 1]] = gate * torch.sigmoid(gate) * (rows @ s["w"][i, n:].double().T)
    return out


def _exact_down(s):
    out = torch.zeros(s["t"], s["n"], dtype=torch.float64, device=DEV)
    at = s["offsets"].tolist()
    weight = s["weights"].reshape(-1).double()
    for i in range(s["e"]):
        j = s["order"][at[i]:at[i + 1]].long()
        out[j // s["top_k"]] += weight[j, None] * (s["x"][at[i]:at[i + 1]].double() @ s["w"][i].double().T)
    return out


def _exact_lora(s):
    out = s["base"].double()
    for i in range(s["adapters"]):
        r = int(s["ranks"][i])
        rows = (s["ids"] == i).nonzero()[:, 0]
        v = s["x"][rows].double() @ s["a"][i, :r].double().T
        out[rows] += float(s["scales"][i]) * (v @ s["b"][i, :, :r].double().T)
    return out
