"""Selection operators of language models, as they are measured: routing to
experts and its gradient, penalties, biases and grammar masks on logits, and
picking the next token from them.

``run`` with ``own`` false computes an operator in elementary torch
operations; with ``own`` true it calls the library.  ``exact`` computes the
same in numpy in 64 bits, from the definitions in ``include/greedy_nms.h``.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one decode step of eight sequences through a layer of 64 experts
        {"name": "route_step", "op": "route", "T": 8, "E": 64, "k": 6, "dtype": "bf16",
         "score": "softmax", "bias": False, "groups": 1, "kept": 1, "top": 1, "renorm": False,
         "scale": 1.0, "masked": False},
        # a decode batch through 256 experts in 8 groups, balanced by a bias
        {"name": "route_batch", "op": "route", "T": 128, "E": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "kept": 4, "top": 2, "renorm": True,
         "scale": 2.5, "masked": False},
        # a long prompt or a training micro-batch through the same layer
        {"name": "route_prompt", "op": "route", "T": 16384, "E": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "kept": 4, "top": 2, "renorm": True,
         "scale": 2.5, "masked": False},
        # an odd number of experts, padded rows and experts switched off
        {"name": "route_ragged", "op": "route", "T": 5003, "E": 60, "k": 4, "dtype": "f16",
         "score": "softmax", "bias": False, "groups": 1, "kept": 1, "top": 1, "renorm": True,
         "scale": 1.0, "masked": True},
        # the gradient of a training micro-batch, weights not renormalised
        {"name": "route_back_softmax", "op": "route_back", "T": 32768, "E": 128, "k": 8,
         "dtype": "bf16", "score": "softmax", "renorm": False, "scale": 1.0},
        # the gradient of renormalised sigmoid weights, an odd batch
        {"name": "route_back_sigmoid", "op": "route_back", "T": 4099, "E": 256, "k": 8,
         "dtype": "f32", "score": "sigmoid", "renorm": True, "scale": 2.5},
        # four chats of a few hundred tokens, logits wanted for a beam search
        {"name": "adjust_few", "op": "adjust", "B": 4, "V": 32000, "L": 300, "dtype": "bf16",
         "bias": 8, "masks": 2},
        # a full decode batch over a large vocabulary
        {"name": "adjust_batch", "op": "adjust", "B": 256, "V": 131072, "L": 2048,
         "dtype": "bf16", "bias": 16, "masks": 64},
        # one chat, almost greedy
        {"name": "pick_one", "op": "pick", "B": 1, "V": 32000, "L": 200, "dtype": "bf16",
         "bias": 0, "masks": 0, "k": 1},
        # a decode batch, an odd vocabulary, float32 logits
        {"name": "pick_batch", "op": "pick", "B": 64, "V": 100003, "L": 1500, "dtype": "f32",
         "bias": 16, "masks": 8, "k": 50},
        # the largest decode batch, many candidates kept
        {"name": "pick_wide", "op": "pick", "B": 256, "V": 131072, "L": 4096, "dtype": "bf16",
         "bias": 16, "masks": 32, "k": 1000},
        # long documents: the history is as long as the vocabulary is wide
        {"name": "pick_long", "op": "pick", "B": 16, "V": 150001, "L": 65536, "dtype": "f16",
         "bias": 300, "masks": 4, "k": 40},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_back", "adjust", "pick", "pick"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("route", "route_back"):
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "route" else 1
        experts = groups * _spread(rng, max(4, 8 // groups), 384 // groups)
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(12, kept * (experts // groups)))
        case = {"op": op, "T": _spread(rng, 1, 4194304 // experts // 2), "E": experts, "k": k,
                "dtype": dtype, "score": rng.choice(["softmax", "sigmoid"]),
                "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5])}
        if op == "route":
            case.update(bias=rng.random() < 0.5, groups=groups, kept=kept,
                        top=rng.choice([1, 2]), masked=rng.random() < 0.3)
        return case
    V = _spread(rng, 500, 200000)
    L = _spread(rng, 1, 40000)
    B = _spread(rng, 1, max(1, min(256, 16000000 // V, 1000000 // L)))
    case = {"op": op, "B": B, "V": V, "L": L, "dtype": dtype, "bias": rng.choice([0, 8, 300]),
            "masks": rng.choice([0, 1, 8])}
    if op == "pick":
        case["k"] = rng.choice([1, _spread(rng, 2, 1000), _spread(rng, 2, 100)])
        case["k"] = min(case["k"], V)
    return case


# ------------------------------------------------------------------ inputs

def _route_inputs(case, g):
    """Router logits: a token prefers a few experts and some experts are
    preferred by most tokens, which the balance bias works against."""
    T, E, dt = case["T"], case["E"], _DTYPES[case["dtype"]]
    dev = "cuda"
    popular = torch.randn(E, generator=g, device=dev) * 0.7
    z = torch.randn(T, E, generator=g, device=dev) * 1.3 + popular
    s = {"live": None, "bias": None}
    if case.get("masked"):
        off = torch.rand(T, E, generator=g, device=dev) < 0.1
        z = torch.where(off, torch.full_like(z, -math.inf), z)
        s["live"] = torch.rand(T, generator=g, device=dev) < 0.9
    s["logits"] = z.to(dt)
    if case.get("bias"):
        s["bias"] = -0.1 * popular + 0.02 * torch.randn(E, generator=g, device=dev)
    return s


def _logit_inputs(case, g):
    """Logits of a decode step: the recent tokens of each row stand out, as
    they do where a model tends to repeat itself; histories repeat common
    tokens; row 0 has just begun."""
    B, V, L, dt = case["B"], case["V"], case["L"], _DTYPES[case["dtype"]]
    dev = "cuda"

    def choice(values):
        at = torch.randint(len(values), (B,), generator=g, device=dev)
        return torch.tensor(values, dtype=torch.float32, device=dev)[at]

    z = torch.randn(B, V, generator=g, device=dev) * 2.5
    common = torch.rand(B, L, generator=g, device=dev) ** 3
    history = (common * V).to(torch.int32).clamp_(0, V - 1)
    length = torch.randint((L + 1) // 2, L + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    prompt = (length * torch.rand(B, generator=g, device=dev)).to(torch.int32)
    if B > 1:
        length[0] = 0
        prompt[0] = 0
    recent = history[:, : min(L, 64)].long()
    z.scatter_(1, recent, z.gather(1, recent) * 0.5 + 5.0)
    s = {"logits": z.to(dt), "history": history, "length": length, "prompt": prompt,
         "repetition": choice([1.0, 1.1, 1.3]), "presence": choice([0.0, 0.5]),
         "frequency": choice([0.0, 0.2, -0.1]), "bias_ids": None, "bias_values": None,
         "allowed": None, "allowed_rows": None}
    M, R = case["bias"], case["masks"]
    if M:
        ids = (torch.rand(B, V, generator=g, device=dev).topk(min(M, V), dim=1).indices
               if V * B < 1 << 22 else
               torch.arange(M, device=dev) * (V // M) +
               torch.randint(max(1, V // M), (B, M), generator=g, device=dev))
        ids = ids.to(torch.int32)
        unused = torch.rand(ids.shape, generator=g, device=dev) < 0.2
        s["bias_ids"] = torch.where(unused, torch.full_like(ids, -1), ids).contiguous()
        s["bias_values"] = torch.randn(ids.shape, generator=g, device=dev) * 3.0
    if R:
        share = torch.rand(R, 1, generator=g, device=dev) ** 2 * 0.9 + 0.05
        words = (V + 63) // 64
        bits = torch.rand(R, words * 64, generator=g, device=dev) < share
        shift = torch.arange(64, device=dev)
        s["allowed"] = (bits.view(R, words, 64).long() << shift).sum(2)
        rows = torch.randint(-R, R, (B,), generator=g, device=dev, dtype=torch.int32)
        s["allowed_rows"] = rows.clamp_(min=-1)
    if case["op"] == "pick":
        k = case["k"]
        s["uniform"] = torch.rand(B, generator=g, device=dev)
        s["temperature"] = choice([0.0, 0.7, 1.0, 1.3])
        s["top_k"] = torch.randint(max(1, k // 2), k + 1, (B,), generator=g, device=dev,
                                   dtype=torch.int32)
        s["top_p"] = choice([0.8, 0.95, 1.0])
        s["min_p"] = choice([0.0, 0.0, 0.02])
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "route":
        s = _route_inputs(case, g)
    elif case["op"] == "route_back":
        s = _route_inputs(case, g)
        # the experts that the forward pass chose, and what came back for them
        s["ids"] = s["logits"].float().topk(case["k"], dim=1).indices.to(torch.int32)
        s["grad"] = torch.randn(case["T"], case["k"], generator=g, device="cuda")
    else:
        s = _logit_inputs(case, g)
        if own:
            # the handle on a batch's rules, which a serving loop keeps while
            # the buffers' contents change from step to step
            import greedy_iou_nms_amd as lib
            s["rules"] = lib.LogitRules(
                case["V"], history=s["history"], history_len=s["length"],
                prompt_len=s["prompt"], repetition=s["repetition"], presence=s["presence"],
                frequency=s["frequency"], bias_ids=s["bias_ids"],
                bias_values=s["bias_values"], allowed=s["allowed"],
                allowed_rows=s["allowed_rows"])
    s["case"] = case
    return s


# ------------------------------------------------------- the plain forms

def _scores(z, kind):
    """Expert scores in 64 bits (choices next to a border decide by them)."""
    z = z.double()
    z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
    if kind == "sigmoid":
        return z, 1.0 / (1.0 + torch.exp(-z))
    top = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return z, e / e.sum(dim=1, keepdim=True)


def _plain_route(s):
    c = s["case"]
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    z, score = _scores(s["logits"], c["score"])
    low = torch.full_like(z, -math.inf)
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(torch.isinf(z), low, choice)
    rank = torch.where(torch.isinf(choice), low, z if s["bias"] is None else choice)
    if G > 1:
        best = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values
        best = best[:, :, : c["top"]]
        some = torch.isinf(best[:, :, 0])
        best = torch.where(torch.isinf(best), torch.zeros_like(best), best).sum(dim=2)
        best = torch.where(some, torch.full_like(best, -math.inf), best)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, G, dtype=torch.bool, device=z.device)
        keep.scatter_(1, order[:, : c["kept"]], True)
        rank = torch.where(keep.repeat_interleave(E // G, dim=1), rank, low)
    if s["live"] is not None:
        rank = torch.where(s["live"][:, None], rank, low)
    rank, ids = torch.sort(rank, dim=1, descending=True, stable=True)
    rank, ids = rank[:, :k], ids[:, :k]
    there = ~torch.isinf(rank)
    w = torch.where(there, score.gather(1, ids), torch.zeros_like(rank))
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    counts = torch.zeros(E + 1, dtype=torch.int32, device=z.device)
    at = torch.where(there, ids, torch.full_like(ids, E)).reshape(-1)
    counts.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    ids = torch.where(there, ids, torch.full_like(ids, -1))
    return {"ids": ids.to(torch.int32), "weights": (w * c["scale"]).float(), "counts": counts[:E]}


def _plain_route_back(s):
    c = s["case"]
    z = s["logits"].float()
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-z))
    else:
        e = torch.exp(z - z.max(dim=1, keepdim=True).values)
        p = e / e.sum(dim=1, keepdim=True)
    at = s["ids"].long()
    chosen = p.gather(1, at)
    g = s["grad"] * c["scale"]
    if c["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        g = (g - (g * chosen).sum(dim=1, keepdim=True) / total) / total
    ds = torch.zeros_like(p).scatter_(1, at, g)
    if c["score"] == "sigmoid":
        dz = ds * p * (1.0 - p)
    else:
        dz = p * (ds - (ds * p).sum(dim=1, keepdim=True))
    return {"grad_logits": dz.to(s["logits"].dtype)}


def _plain_adjusted(s):
    """The adjusted logits in float32, one rounding a step."""
    z = s["logits"].float()
    B, V = z.shape
    L = s["history"].shape[1]
    at = torch.arange(L, device=z.device)
    inside = at < s["length"][:, None]
    generated = inside & (at >= s["prompt"][:, None])
    token = s["history"].long()
    count = torch.zeros(B, V + 1, dtype=torch.int32, device=z.device)
    count.scatter_add_(1, torch.where(generated, token, V), torch.ones_like(s["history"]))
    seen = torch.zeros(B, V + 1, dtype=torch.bool, device=z.device)
    seen.scatter_(1, torch.where(inside, token, V), True)
    count, seen = count[:, :V], seen[:, :V]
    r = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
    z = torch.where(count > 0, z - s["frequency"][:, None] * count.float(), z)
    z = torch.where(count > 0, z - s["presence"][:, None], z)
    if s["bias_ids"] is not None:
        ids = s["bias_ids"].long()
        bias = torch.zeros(B, V + 1, device=z.device)
        bias.scatter_(1, torch.where(ids < 0, V, ids), s["bias_values"])
        z = z + bias[:, :V]
    if s["allowed"] is not None:
        v = torch.arange(V, device=z.device)
        bits = ((s["allowed"][:, v >> 6] >> (v & 63)) & 1).bool()
        rows = s["allowed_rows"].long()
        ok = bits[rows.clamp(min=0)] | (rows < 0)[:, None]
        z = torch.where(ok, z, torch.full_like(z, -math.inf))
    return z


def _plain_pick(s):
    z = _plain_adjusted(s)
    k = s["case"]["k"]
    cand, order = torch.sort(z, dim=1, descending=True, stable=True)
    cand, order = cand[:, :k].double(), order[:, :k]
    heat = s["temperature"].double()[:, None]
    warm = torch.where(heat > 0, heat, torch.ones_like(heat))
    at = torch.arange(k, device=z.device)
    there = (at < s["top_k"][:, None]) & ~torch.isinf(cand)
    w = torch.where(there, torch.exp((cand - cand[:, :1]) / warm), torch.zeros_like(cand))
    cum = torch.cumsum(w, dim=1)
    # the shortest prefix that holds top_p of the weight, at least one
    short = (cum < s["top_p"].double()[:, None] * cum[:, -1:]).sum(dim=1) + 1
    large = (there & (w >= s["min_p"].double()[:, None])).sum(dim=1)
    n = torch.minimum(torch.minimum(short, large), there.sum(dim=1)).clamp(min=1)
    total = cum.gather(1, n[:, None] - 1)
    j = (cum <= s["uniform"].double()[:, None] * total).sum(dim=1)
    j = torch.where(heat[:, 0] > 0, torch.minimum(j, n - 1), torch.zeros_like(j))[:, None]
    e = torch.exp((z.double() - cand[:, :1]) / warm).sum(dim=1, keepdim=True)
    logprob = (cand.gather(1, j) - cand[:, :1]) / warm - torch.log(e)
    return {"ids": order.gather(1, j)[:, 0].to(torch.int32), "logprobs": logprob[:, 0].float()}


def run(state):
    c = state["case"]
    if own:
        import greedy_iou_nms_amd as lib
        if c["op"] == "route":
            ids, weights, counts = lib.route_experts(
                state["logits"], c["k"], score=c["score"], bias=state["bias"],
                groups=c["groups"], kept_groups=c["kept"], group_top=c["top"],
                renormalise=c["renorm"], scale=c["scale"], live=state["live"], counts=True)
            return {"ids": ids, "weights": weights, "counts": counts}
        if c["op"] == "route_back":
            return {"grad_logits": lib.route_experts_backward(
                state["logits"], state["ids"], state["grad"], score=c["score"],
                renormalise=c["renorm"], scale=c["scale"])}
        if c["op"] == "adjust":
            return {"logits": lib.adjust_logits(state["logits"], state["rules"])}
        ids, logprobs = lib.pick_tokens(
            state["logits"], state["uniform"], max_top_k=c["k"], temperature=state["temperature"],
            top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"],
            rules=state["rules"])
        return {"ids": ids, "logprobs": logprobs}
    if c["op"] == "route":
        return _plain_route(state)
    if c["op"] == "route_back":
        return _plain_route_back(state)
    if c["op"] == "adjust":
        return {"logits": _plain_adjusted(state).to(state["logits"].dtype)}
    return _plain_pick(state)


def work(case):
    if case["op"] in ("route", "route_back"):
        T, E, k, z = case["T"], case["E"], case["k"], _SIZE[case["dtype"]]
        if case["op"] == "route":
            # exp, add, compare per expert; a quotient per chosen one
            return {"bytes": T * E * z + T * k * 8 + E * 4 * (1 + bool(case["bias"])),
                    "flops": T * (4 * E + 3 * k)}
        if case["score"] == "softmax" and not case["renorm"]:
            return {"bytes": 2 * T * E * z + T * k * 8, "flops": T * (6 * E + 6 * k)}
        # the gradient is zero but for the chosen experts, and needs only their logits
        return {"bytes": T * E * z + T * k * (8 + z), "flops": T * 12 * k}
    B, V, L, z = case["B"], case["V"], case["L"], _SIZE[case["dtype"]]
    # lengths are between half of L and L
    read = B * V * z + B * L * 3 + case["masks"] * ((V + 63) // 64) * 8 + B * case["bias"] * 8
    if case["op"] == "adjust":
        return {"bytes": read + B * V * z, "flops": B * (V + 2 * L)}
    return {"bytes": read + B * 36, "flops": B * (4 * V + 2 * L)}


# ------------------------------------- the definitions, in 64 bits, in numpy

def _host(t):
    return None if t is None else (t.double() if t.is_floating_point() else t).cpu().numpy()


def _exact_route(c, s):
    z, live = _host(s["logits"]), _host(s["live"])
    T, E = z.shape
    k, G = c["k"], c["groups"]
    with np.errstate(over="ignore"):
        if c["score"] == "sigmoid":
            score = 1.0 / (1.0 + np.exp(-z))
        else:
            score = np.exp(z - z.max(axis=1, keepdims=True))
            score /= score.sum(axis=1, keepdims=True)
    bias = _host(s["bias"])
    choice = score if bias is None else score + bias
    out = np.isneginf(z) if live is None else np.isneginf(z) | ~live[:, None]
    choice = np.where(out, -np.inf, choice)
    if G > 1:
        parts = -np.sort(-choice.reshape(T, G, E // G), axis=2)[:, :, : c["top"]]
        total = np.where(np.isneginf(parts), 0.0, parts).sum(axis=2)
        total[np.isneginf(parts[:, :, 0])] = -np.inf
        place = np.argsort(np.argsort(-total, axis=1, kind="stable"), axis=1)
        out = out | np.repeat(place >= c["kept"], E // G, axis=1)
    rank = np.where(out, -np.inf, z if bias is None else choice)
    ids = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    there = ~np.take_along_axis(out, ids, axis=1)
    w = np.where(there, np.take_along_axis(score, ids, axis=1), 0.0)
    if c["renorm"]:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return {"ids": np.where(there, ids, -1).astype(np.int32), "weights": w * c["scale"],
            "counts": np.bincount(ids[there], minlength=E).astype(np.int32)}


def _exact_route_back(c, s):
    # the gradient by the Jacobian of the weights, expert by expert
    z, ids, g = _host(s["logits"]), _host(s["ids"]), _host(s["grad"]) * c["scale"]
    rows = np.arange(z.shape[0])[:, None]
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + np.exp(-z))
    else:
        p = np.exp(z - z.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
    q = p[rows, ids]
    if c["renorm"]:
        share = q / q.sum(axis=1, keepdims=True)
        inner = (g * share).sum(axis=1, keepdims=True)
        # d share_i / d q_j = ([i = j] - share_i) / sum q
        dq = (g - inner) / q.sum(axis=1, keepdims=True)
    else:
        dq = g
    dz = np.zeros_like(z)
    if c["score"] == "sigmoid":
        dz[rows, ids] = dq * q * (1.0 - q)
    else:
        dz -= p * (dq * q).sum(axis=1, keepdims=True)
        dz[rows, ids] += dq * q
    return {"grad_logits": dz}


def _exact_adjusted(s):
    """Each step in 64 bits, rounded to float32 as the definition says."""
    z = _host(s["logits"])
    B, V = z.shape
    history, length, prompt = _host(s["history"]), _host(s["length"]), _host(s["prompt"])
    r, f, p = _host(s["repetition"]), _host(s["frequency"]), _host(s["presence"])
    ids, values = _host(s["bias_ids"]), _host(s["bias_values"])
    allowed, rows = _host(s["allowed"]), _host(s["allowed_rows"])

    def once(x):
        return x.astype(np.float32).astype(np.float64)

    for b in range(B):
        seen = np.unique(history[b, : length[b]])
        x = z[b, seen]
        x = once(np.where(x > 0, x / r[b], x * r[b]))
        z[b, seen] = x
        token, times = np.unique(history[b, prompt[b]: length[b]], return_counts=True)
        z[b, token] = once(once(z[b, token] - once(f[b] * times)) - p[b])
        if ids is not None:
            used = ids[b] >= 0
            z[b, ids[b][used]] = once(z[b, ids[b][used]] + values[b][used])
        if allowed is not None and rows[b] >= 0:
            bits = np.unpackbits(allowed[rows[b]].view(np.uint8), bitorder="little")[:V]
            z[b, bits == 0] = -np.inf
    return z


def _exact_pick(c, s):
    z = _exact_adjusted(s)
    u, heat = _host(s["uniform"]), _host(s["temperature"])
    top_k, top_p, min_p = _host(s["top_k"]), _host(s["top_p"]), _host(s["min_p"])
    ids, logprobs = np.empty(len(z), np.int32), np.empty(len(z))
    for b, x in enumerate(z):
        k = int(min(top_k[b], np.isfinite(x).sum()))
        # the k largest values, and by index those that are equal to the last
        edge = np.partition(x, x.size - k)[x.size - k]
        at = np.flatnonzero(x >= edge)
        at = at[np.argsort(-x[at], kind="stable")][:k]
        t = heat[b] if heat[b] > 0 else 1.0
        w = np.exp((x[at] - x[at[0]]) / t)
        cum = np.cumsum(w)
        n = min(int(np.searchsorted(cum, top_p[b] * cum[-1])) + 1, int((w >= min_p[b]).sum()), k)
        n = max(n, 1)
        j = min(int(np.searchsorted(cum[:n], u[b] * cum[n - 1], side="right")), n - 1)
        j = j if heat[b] > 0 else 0
        ids[b] = at[j]
        logprobs[b] = (x[at[j]] - x[at[0]]) / t - np.log(np.exp((x - x[at[0]]) / t).sum())
    return {"ids": ids, "logprobs": logprobs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "route_back":
        return _exact_route_back(case, s)
    if case["op"] == "adjust":
        return {"logits": _exact_adjusted(s)}
    return _exact_pick(case, s)
