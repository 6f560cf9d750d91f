"""Training operators of language models, as they are measured: log
probabilities of given tokens, the clipped policy loss and the preference loss
that are made of them, and the balance loss of routing, with their gradients.

``run`` with ``own`` false computes an operator in elementary torch
operations; with ``own`` true it calls the library.  ``exact`` computes the
same in 64 bits, from the definitions.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # the chosen tokens of one decode step, scored under a second model
        {"name": "logprobs_step", "op": "logprobs", "T": 8, "V": 32000, "dtype": "bf16",
         "heat": True, "entropy": False, "train": False, "masked": 0.0},
        # a long prompt scored token by token, with the entropies
        {"name": "logprobs_prompt", "op": "logprobs", "T": 4097, "V": 131072, "dtype": "bf16",
         "heat": False, "entropy": True, "train": False, "masked": 0.0},
        # a user's own loss on log probabilities and entropies: there and back
        {"name": "logprobs_train", "op": "logprobs", "T": 1999, "V": 100003, "dtype": "f32",
         "heat": False, "entropy": True, "train": True, "masked": 0.2},
        # the policy step of a small micro-batch
        {"name": "policy_small", "op": "policy", "T": 64, "V": 32000, "dtype": "bf16",
         "heat": False, "entropy": False, "kl": 0.0, "autograd": False, "masked": 0.3},
        # the policy step of a large micro-batch over a large vocabulary, KL term included
        {"name": "policy_batch", "op": "policy", "T": 4096, "V": 131072, "dtype": "bf16",
         "heat": False, "entropy": False, "kl": 0.04, "autograd": False, "masked": 0.1},
        # an odd vocabulary, sampled at several temperatures, an entropy bonus, through autograd
        {"name": "policy_ragged", "op": "policy", "T": 1003, "V": 150001, "dtype": "f16",
         "heat": True, "entropy": True, "kl": 0.04, "autograd": True, "masked": 0.2},
        # two short pairs
        {"name": "preference_short", "op": "preference", "P": 2, "T": 237, "V": 32000,
         "dtype": "f32", "kind": "sigmoid", "average": False, "masked": 0.3},
        # a batch of pairs, their prompts masked
        {"name": "preference_pairs", "op": "preference", "P": 8, "T": 8192, "V": 32000,
         "dtype": "bf16", "kind": "sigmoid", "average": False, "masked": 0.4},
        # long answers over a large vocabulary, judged by their mean log probability
        {"name": "preference_long", "op": "preference", "P": 2, "T": 4001, "V": 131072,
         "dtype": "bf16", "kind": "squared", "average": True, "masked": 0.2},
        # a small micro-batch through a layer of 64 experts
        {"name": "balance_step", "op": "balance", "T": 512, "E": 64, "k": 6, "dtype": "bf16",
         "score": "softmax", "z": 0.0, "S": 1, "masked": 0.0},
        # a training micro-batch through 256 experts, balanced within each sequence
        {"name": "balance_batch", "op": "balance", "T": 16384, "E": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "z": 0.0, "S": 16, "masked": 0.0},
        # an odd number of experts and of tokens, padded rows, the z term
        {"name": "balance_ragged", "op": "balance", "T": 65521, "E": 60, "k": 4, "dtype": "f16",
         "score": "softmax", "z": 0.001, "S": 1, "masked": 0.1},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "policy", "policy", "preference", "balance"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    masked = rng.choice([0.0, rng.uniform(0.05, 0.6)])
    if op == "balance":
        experts = _spread(rng, 4, 512)
        tokens = _spread(rng, 16, 1 << 17)
        return {"op": op, "T": tokens, "E": experts, "k": rng.randint(1, min(12, experts)),
                "dtype": dtype, "score": rng.choice(["softmax", "sigmoid"]),
                "z": rng.choice([0.0, 0.001]), "S": rng.choice([1, _spread(rng, 1, 64)]),
                "masked": masked}
    V = _spread(rng, 500, 200000)
    most = (1 << 29) // (_SIZE[dtype] * V)
    case = {"op": op, "T": _spread(rng, 1, min(16384, most)), "V": V, "dtype": dtype,
            "masked": masked}
    if op == "logprobs":
        case.update(heat=rng.random() < 0.5, entropy=rng.random() < 0.5, train=rng.random() < 0.5)
    elif op == "policy":
        case.update(heat=rng.random() < 0.3, entropy=rng.random() < 0.3,
                    kl=rng.choice([0.0, 0.04]), autograd=rng.random() < 0.3)
    else:
        case["T"] = max(case["T"], min(most, 32))
        case.update(P=_spread(rng, 1, max(1, min(32, case["T"] // 8))),
                    kind=rng.choice(["sigmoid", "hinge", "squared"]),
                    average=rng.random() < 0.4)
    return case


# ------------------------------------------------------------------ inputs

_CLIP, _CLIP_HIGH, _BONUS, _BETA, _SMOOTHING, _BALANCE = 0.2, 0.28, 0.01, 0.1, 0.05, 0.01


def _borders(T, n, g):
    """n ragged pieces of T rows, the first ones at least a row long."""
    cut = torch.rand(n - 1, generator=g, device="cuda").sort().values
    even = torch.arange(1, n, device="cuda") / n
    inner = (T * (0.5 * even + 0.5 * cut)).long()
    ends = torch.tensor([0, T], device="cuda")
    return torch.cat([ends[:1], inner, ends[1:]]).to(torch.int64)


def _loss_scale(case):
    """float16 gradients are of a scaled loss, as in mixed precision training:
    a power of two that brings them into float16's range."""
    if case["dtype"] != "f16":
        return None
    shares = {"balance": case["T"] * case.get("E", 1) / 4, "preference": 1.0}.get(
        case["op"], case["T"])
    if case.get("average"):
        shares = case["T"] / (2 * case["P"])
    return torch.tensor(2.0 ** round(math.log2(64 * shares)), device="cuda")


def _logit_inputs(case, g):
    """Logits of a model on its own text: the next token stands out among
    many that are far below it."""
    T, V, dev = case["T"], case["V"], "cuda"
    f32 = torch.float32
    z = torch.randn(T, V, generator=g, device=dev)
    z *= 2.5
    token = (torch.rand(T, generator=g, device=dev) * V).long().clamp_(max=V - 1)
    level = math.log(V) + 3.0 + 2.0 * torch.randn(T, 1, generator=g, device=dev)
    z.scatter_(1, token[:, None], level)
    # what the sampler took down, a few steps of training ago
    lp = level[:, 0] - (z.exp().sum(dim=1)).log()
    s = {"logits": z.to(_DTYPES[case["dtype"]]), "scale": _loss_scale(case)}
    out = torch.rand(T, generator=g, device=dev) < case["masked"]
    s["tokens"] = torch.where(out, torch.full_like(token, -1), token).to(torch.int32)
    noise = torch.randn(3, T, generator=g, device=dev)
    s["heat"] = None
    if case.get("heat"):
        s["heat"] = 0.7 + 0.6 * torch.rand(T, generator=g, device=dev)
    if case["op"] == "logprobs" and case["train"]:
        up = 1.0 if s["scale"] is None else s["scale"]
        s["grad"], s["grad_entropy"] = noise[0] * up / T, noise[1] * up / T
    elif case["op"] == "policy":
        s["old"] = lp + 0.2 * noise[0]
        s["ref"] = lp + 0.4 * noise[1] if case["kl"] else None
        s["advantages"] = noise[2] + 0.3
        s["weights"] = (~out).to(f32) / (~out).sum().clamp(min=1)
        s["tokens"] = token.to(torch.int32)
    elif case["op"] == "preference":
        s["offsets"] = _borders(T, 2 * case["P"], g)
        at = torch.arange(T, device=dev)
        owner = (s["offsets"][None, 1:-1] <= at[:, None]).sum(dim=1)
        ref = torch.zeros(2 * case["P"], dtype=torch.float64, device=dev)
        n = torch.zeros_like(ref)
        ref.index_add_(0, owner, torch.where(out, 0.0, (lp + 0.2 * noise[0]).double()))
        n.index_add_(0, owner, (~out).double())
        s["ref"] = (ref / n.clamp(min=1) if case["average"] else ref).float()
    return s


def _route_inputs(case, g):
    """Router logits: some experts are preferred by most tokens."""
    T, E, dev = case["T"], case["E"], "cuda"
    popular = torch.randn(E, generator=g, device=dev) * 0.7
    z = torch.randn(T, E, generator=g, device=dev) * 1.3 + popular
    s = {"logits": z.to(_DTYPES[case["dtype"]]), "live": None, "offsets": None,
         "scale": _loss_scale(case)}
    if case["masked"]:
        s["live"] = torch.rand(T, generator=g, device=dev) >= case["masked"]
    if case["S"] > 1:
        s["offsets"] = _borders(T, case["S"], g)
    # the experts that the router chose
    s["ids"] = s["logits"].float().topk(case["k"], dim=1).indices.to(torch.int32).contiguous()
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = _route_inputs(case, g) if case["op"] == "balance" else _logit_inputs(case, g)
    s["case"] = case
    return s


# ------------------------------------------------------- the plain forms

def _softmax(z):
    """Probabilities, and the logits less the logarithm of their exponentials'
    sum: a matrix less a column in 64 bits, for sums over many rows."""
    z = z - z.max(dim=1, keepdim=True).values
    e = torch.exp(z)
    total = e.sum(dim=1, keepdim=True, dtype=torch.float64)
    return e / total.float(), z, torch.log(total)


def _plain_rows(s):
    """Which rows count, their tokens, all probabilities and log
    probabilities, and the tokens' log probabilities in 64 bits."""
    z = s["logits"].float()
    if s["heat"] is not None:
        z = z / s["heat"][:, None]
    p, z, log_total = _softmax(z)
    token = s["tokens"].long()
    used = (token >= 0) & (token < z.shape[1])
    if s.get("weights") is not None:
        used = used & (s["weights"] != 0)
    token = torch.where(used, token, torch.zeros_like(token))
    lp = (z.gather(1, token[:, None]).double() - log_total)[:, 0]
    return used, token, p, z - log_total.float(), torch.where(used, lp, torch.zeros_like(lp))


def _plain_entropy(used, p, logp):
    h = -(p * logp).sum(dim=1)
    return torch.where(used, h, torch.zeros_like(h))


def _plain_grad(s, used, token, p, logp, up, d_lp, h=None, d_h=None):
    """The gradient in the logits of up times what has d_lp in the token's log
    probability and d_h in the entropy."""
    up = 1.0 if up is None else up
    d_lp = torch.where(used, d_lp * up, torch.zeros_like(d_lp))
    dz = p * -d_lp[:, None]
    dz.scatter_add_(1, token[:, None], d_lp[:, None])
    if d_h is not None:
        d_h = torch.where(used, d_h * up, torch.zeros_like(d_h))
        dz = dz - d_h[:, None] * p * (logp + h[:, None])
    if s["heat"] is not None:
        dz = dz / s["heat"][:, None]
    return dz.to(s["logits"].dtype)


def _plain_logprobs(s):
    c = s["case"]
    used, token, p, logp, lp = _plain_rows(s)
    out = {"logprobs": lp.float()}
    h = None
    if c["entropy"]:
        h = out["entropies"] = _plain_entropy(used, p, logp)
    if c["train"]:
        out["grad_logits"] = _plain_grad(s, used, token, p, logp, None, s["grad"],
                                         h, s["grad_entropy"] if c["entropy"] else None)
    return out


def _plain_policy(s):
    c = s["case"]
    used, token, p, logp, lp = _plain_rows(s)
    lp = lp.float()
    w, a = s["weights"], s["advantages"]
    r = torch.exp(lp - s["old"])
    free, held = r * a, r.clamp(1.0 - _CLIP, 1.0 + _CLIP_HIGH) * a
    each = -torch.minimum(free, held)
    d_lp = torch.where(free <= held, -free, torch.zeros_like(free))
    if c["kl"]:
        q = s["ref"] - lp
        each = each + c["kl"] * (torch.exp(q) - q - 1.0)
        d_lp = d_lp + c["kl"] * (1.0 - torch.exp(q))
    out = {"logprobs": lp}
    h = d_h = None
    if c["entropy"]:
        h = out["entropies"] = _plain_entropy(used, p, logp)
        each = each - _BONUS * h
        d_h = -_BONUS * w
    each = torch.where(used, w * each, torch.zeros_like(each))
    out["loss"] = each.double().sum().float()
    out["grad_logits"] = _plain_grad(s, used, token, p, logp, s["scale"], w * d_lp, h, d_h)
    return out


def _plain_preference(s):
    c = s["case"]
    P, T = c["P"], c["T"]
    s = dict(s, heat=None)
    used, token, p, logp, lp = _plain_rows(s)
    at = torch.arange(T, device=lp.device)
    owner = (s["offsets"][None, 1:-1] <= at[:, None]).sum(dim=1)
    total = torch.zeros(2 * P, dtype=torch.float64, device=lp.device)
    total = total.index_add(0, owner, lp)
    n = torch.ones_like(total)
    if c["average"]:
        n = torch.zeros_like(total).index_add(0, owner, used.double()).clamp(min=1.0)
    total = total / n
    rel = total - s["ref"].double()
    h = _BETA * (rel[:P] - rel[P:])
    if c["kind"] == "sigmoid":
        e = _SMOOTHING
        # log(1 + exp(-h)) and log(1 + exp(h))
        below = torch.log(1.0 + torch.exp(-h.abs()))
        each = (1.0 - e) * (below + (-h).clamp(min=0)) + e * (below + h.clamp(min=0))
        d_h = 1.0 / (1.0 + torch.exp(-h)) - (1.0 - e)
    elif c["kind"] == "hinge":
        each = (1.0 - h).clamp(min=0)
        d_h = -(h < 1.0).double()
    else:
        each = ((h - 0.5) / _BETA) ** 2
        d_h = 2.0 * (h - 0.5) / _BETA ** 2
    d_h = d_h * (_BETA / P)
    d_lp = (torch.cat([d_h, -d_h]) / n).float()[owner]
    return {"loss": (each.sum() / P).float(), "logprobs": total.float(), "margins": h.float(),
            "grad_logits": _plain_grad(s, used, token, p, logp, s["scale"], d_lp)}


def _plain_balance(s):
    c = s["case"]
    T, E, S = c["T"], c["E"], c["S"]
    z = s["logits"].float()
    live = torch.ones(T, device=z.device) if s["live"] is None else s["live"].float()
    if s["offsets"] is None:
        owner = torch.zeros(T, dtype=torch.int64, device=z.device)
    else:
        at = torch.arange(T, device=z.device)
        owner = (s["offsets"][None, 1:-1] <= at[:, None]).sum(dim=1)
    at = owner[:, None] * E + s["ids"].long()
    at = torch.where(live[:, None] > 0, at, torch.full_like(at, S * E)).reshape(-1)
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device=z.device)
    counts.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    counts = counts[: S * E].view(S, E)
    tokens = torch.zeros(S, device=z.device).index_add(0, owner, live)
    share = counts.float() / counts.sum(dim=1, keepdim=True).clamp(min=1).float() * E
    a = (_BALANCE / S) * share / tokens.clamp(min=1.0)[:, None]
    a = a[owner] * live[:, None]
    p, below, log_total = _softmax(z)
    if c["score"] == "sigmoid":
        sig = 1.0 / (1.0 + torch.exp(-z))
        total = sig.sum(dim=1, keepdim=True)
        inner = (a * sig).sum(dim=1, keepdim=True) / total
        dz = sig * (1.0 - sig) / total * (a - inner)
    else:
        inner = (a * p).sum(dim=1, keepdim=True)
        dz = p * (a - inner)
    each = inner[:, 0]
    if c["z"]:
        lse = (z[:, 0] - below[:, 0]) + log_total.float()[:, 0]
        w = c["z"] / live.sum().clamp(min=1.0) * live
        each = each + w * lse * lse
        dz = dz + (2.0 * w * lse)[:, None] * p
    if s["scale"] is not None:
        dz = dz * s["scale"]
    return {"loss": each.double().sum().float(), "counts": counts if S > 1 else counts[0],
            "grad_logits": dz.to(s["logits"].dtype)}


def run(state):
    c = state["case"]
    if not own:
        return {"logprobs": _plain_logprobs, "policy": _plain_policy,
                "preference": _plain_preference, "balance": _plain_balance}[c["op"]](state)
    import greedy_iou_nms_amd as lib
    z = state["logits"]
    if c["op"] == "logprobs":
        z = z.detach().requires_grad_(c["train"])
        got = lib.token_logprobs(z, state["tokens"], temperature=state["heat"],
                                 entropy=c["entropy"])
        out = dict(zip(("logprobs", "entropies"), got if c["entropy"] else (got,)))
        if c["train"]:
            given = (state["grad"], state["grad_entropy"]) if c["entropy"] else (state["grad"],)
            torch.autograd.backward(tuple(out.values()), given)
            out = {k: v.detach() for k, v in out.items()}
            out["grad_logits"] = z.grad
        return out
    if c["op"] == "policy":
        rest = dict(weights=state["weights"], ref_logprobs=state["ref"],
                    temperature=state["heat"], clip=_CLIP, clip_high=_CLIP_HIGH, kl=c["kl"],
                    entropy=_BONUS if c["entropy"] else None)
        if c["autograd"]:
            z = z.detach().requires_grad_()
            got = lib.policy_loss(z, state["tokens"], state["old"], state["advantages"], **rest)
            got[0].backward(state["scale"])
            got = (got[0].detach(), z.grad) + got[1:]
        else:
            got = lib.policy_loss_with_grad(z, state["tokens"], state["old"],
                                            state["advantages"],
                                            grad_loss=state["scale"], **rest)
        return dict(zip(("loss", "grad_logits", "logprobs", "entropies"), got))
    if c["op"] == "preference":
        got = lib.preference_loss_with_grad(
            z, state["tokens"], state["offsets"], ref_logprobs=state["ref"], beta=_BETA,
            kind=c["kind"], smoothing=_SMOOTHING if c["kind"] == "sigmoid" else 0.0,
            average=c["average"], grad_loss=state["scale"])
        return dict(zip(("loss", "grad_logits", "logprobs", "margins"), got))
    got = lib.balance_loss_with_grad(z, state["ids"], score=c["score"], balance=_BALANCE,
                                     z=c["z"], offsets=state["offsets"], live=state["live"],
                                     grad_loss=state["scale"])
    return dict(zip(("loss", "grad_logits", "counts"), got))


def work(case):
    T, z = case["T"], _SIZE[case["dtype"]]
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        live = T * (1.0 - case["masked"])
        # max, exp, sum, the inner product and the gradient's four per expert
        return {"bytes": int(live * E * z + T * E * z + live * k * 4 + 4 * case["S"] * E),
                "flops": int(live * E * 9)}
    V = case["V"]
    # rows that do not count need not be read; the gradient is written for all
    live = T * (1.0 - case["masked"])
    train = case.get("train", True)
    side = {"logprobs": 12, "policy": 28, "preference": 4}[case["op"]]
    more = 3 if case.get("entropy") else 0
    # max, subtract, exp, add; and of the gradient exp, multiply, subtract
    return {"bytes": int(live * V * z + train * T * V * z + T * side),
            "flops": int(live * V * (4 + more + train * (3 + more)))}


# ------------------------------------------------- the definitions, in 64 bits

def _exact_rows(s, weigh):
    """A few rows at a time: log softmax in 64 bits, and what `weigh` makes of
    the rows at `at`: the gradients in the token's log probability and in the
    entropy.  Returns the tokens' log probabilities, entropies and the gradient
    in the logits (None where `weigh` is)."""
    z = s["logits"]
    T, V = z.shape
    used = s["tokens"] >= 0
    if s.get("weights") is not None:
        used = used & (s["weights"] != 0)
    lp = torch.zeros(T, dtype=torch.float64, device=z.device)
    h = torch.zeros_like(lp)
    dz = torch.zeros(T, V, dtype=torch.float64, device=z.device) if weigh else None
    rows = torch.nonzero(used)[:, 0]
    for at in rows.split(max(1, (1 << 26) // V)):
        t = 1.0 if s["heat"] is None else s["heat"][at].double()[:, None]
        y = torch.log_softmax(z[at].double() / t, dim=1)
        token = s["tokens"][at].long()
        mine = y[torch.arange(len(at), device=z.device), token]
        p = y.exp()
        ent = -torch.where(p > 0, p * y, torch.zeros_like(p)).sum(dim=1)
        lp[at], h[at] = mine, ent
        if weigh:
            d_lp, d_h = weigh(at, mine, ent)
            one = torch.zeros_like(p)
            one[torch.arange(len(at), device=z.device), token] = 1.0
            # d lp / d z_j = ([j = token] - p_j) / t; d h / d z_j = -p_j (log p_j + h) / t
            g = d_lp[:, None] * (one - p)
            if d_h is not None:
                g -= d_h[:, None] * p * (y + ent[:, None])
            dz[at] = g / t
    return lp, h, dz


def _upstream(s):
    return 1.0 if s["scale"] is None else float(s["scale"])


def _exact_logprobs(c, s):
    def weigh(at, mine, ent):
        return s["grad"][at].double(), s["grad_entropy"][at].double() if c["entropy"] else None

    lp, h, dz = _exact_rows(s, weigh if c["train"] else None)
    out = {"logprobs": lp}
    if c["entropy"]:
        out["entropies"] = h
    if c["train"]:
        out["grad_logits"] = dz
    return out


def _exact_policy(c, s):
    w, adv, old = s["weights"].double(), s["advantages"].double(), s["old"].double()
    total = []

    def weigh(at, mine, ent):
        r = (mine - old[at]).exp()
        a = adv[at]
        # the objective stops growing past the clip on the advantage's side
        stopped = ((a > 0) & (r > 1 + _CLIP_HIGH)) | ((a < 0) & (r < 1 - _CLIP))
        each = -a * torch.where(stopped, torch.where(a > 0, 1 + _CLIP_HIGH, 1 - _CLIP), r)
        d = torch.where(stopped, torch.zeros_like(r), -a * r)
        if c["kl"]:
            q = s["ref"][at].double() - mine
            each = each + c["kl"] * (torch.expm1(q) - q)
            d = d - c["kl"] * torch.expm1(q)
        if c["entropy"]:
            each = each - _BONUS * ent
        total.append((w[at] * each).sum())
        up = _upstream(s)
        return up * w[at] * d, -up * _BONUS * w[at] if c["entropy"] else None

    lp, h, dz = _exact_rows(s, weigh)
    loss = sum(total) if total else torch.zeros((), dtype=torch.float64, device=w.device)
    out = {"logprobs": lp}
    if c["entropy"]:
        out["entropies"] = h
    out.update(loss=loss, grad_logits=dz)
    return out


def _exact_preference(c, s):
    s = dict(s, heat=None)
    P = c["P"]
    lp, _, _ = _exact_rows(s, None)
    ends = s["offsets"].tolist()
    used = s["tokens"] >= 0
    sums, sizes = [], []
    for b, e in zip(ends[:-1], ends[1:]):
        n = max(1, int(used[b:e].sum())) if c["average"] else 1
        sums.append(float(lp[b:e].sum()) / n)
        sizes.append(n)
    ref = s["ref"].double().tolist()
    loss, margins, slope = 0.0, [], [0.0] * (2 * P)
    for i in range(P):
        h = _BETA * ((sums[i] - ref[i]) - (sums[P + i] - ref[P + i]))
        margins.append(h)
        if c["kind"] == "sigmoid":
            up = math.log1p(math.exp(-abs(h))) + max(-h, 0.0)
            down = math.log1p(math.exp(-abs(h))) + max(h, 0.0)
            loss += ((1 - _SMOOTHING) * up + _SMOOTHING * down) / P
            d = -(1 - _SMOOTHING) * math.exp(-down) + _SMOOTHING * math.exp(-up)
        elif c["kind"] == "hinge":
            loss += max(0.0, 1 - h) / P
            d = -1.0 if h < 1 else 0.0
        else:
            loss += (h / _BETA - 0.5 / _BETA) ** 2 / P
            d = 2 * (h / _BETA - 0.5 / _BETA) / _BETA
        slope[i], slope[P + i] = d * _BETA / P / sizes[i], -d * _BETA / P / sizes[P + i]
    f64 = torch.float64
    per_row = torch.zeros_like(lp)
    for q, (b, e) in enumerate(zip(ends[:-1], ends[1:])):
        per_row[b:e] = slope[q] * _upstream(s)
    _, _, dz = _exact_rows(s, lambda at, mine, ent: (per_row[at], None))
    dev = lp.device
    return {"loss": torch.tensor(loss, dtype=f64, device=dev),
            "logprobs": torch.tensor(sums, dtype=f64, device=dev),
            "margins": torch.tensor(margins, dtype=f64, device=dev), "grad_logits": dz}


def _exact_balance(c, s):
    z = s["logits"].double()
    T, E, S = c["T"], c["E"], c["S"]
    dev = z.device
    live = torch.ones(T, dtype=torch.bool, device=dev) if s["live"] is None else s["live"]
    ends = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    score = torch.softmax(z, dim=1)
    if c["score"] == "sigmoid":
        sig = torch.sigmoid(z)
        score = sig / sig.sum(dim=1, keepdim=True)
    loss = torch.zeros((), dtype=torch.float64, device=dev)
    counts = torch.zeros(S, E, dtype=torch.int32, device=dev)
    dz = torch.zeros_like(z)
    for q, (b, e) in enumerate(zip(ends[:-1], ends[1:])):
        rows = torch.nonzero(live[b:e])[:, 0] + b
        n = len(rows)
        counts[q] = torch.bincount(s["ids"][rows].long().reshape(-1), minlength=E)
        if n == 0:
            continue
        f = E * counts[q].double() / counts[q].sum()
        mean = score[rows].sum(dim=0) / n
        loss = loss + _BALANCE / S * (f * mean).sum()
        # d mean_e / d z_j = score_e ([e = j] - score_j) / n, less (1 - sigmoid_j) for sigmoids
        d = score[rows] * (f - (score[rows] * f).sum(dim=1, keepdim=True)) / n
        if c["score"] == "sigmoid":
            d = d * (1.0 - sig[rows])
        dz[rows] = _BALANCE / S * d
    if c["z"] and bool(live.any()):
        lse = torch.logsumexp(z[live], dim=1)
        loss = loss + c["z"] * (lse * lse).mean()
        dz[live] += c["z"] * 2.0 / len(lse) * lse[:, None] * torch.softmax(z[live], dim=1)
    return {"loss": loss, "counts": counts if S > 1 else counts[0],
            "grad_logits": dz * _upstream(s)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "policy": _exact_policy,
            "preference": _exact_preference, "balance": _exact_balance}[case["op"]](case, s)
