"""A sparse layer's operators: what is measured of them, and their plain form.

Three operators of a layer whose tokens each go to a few of many experts:

* routing: a token's logits over E experts -> its top_k experts and their weights.
  Scores are softmax(logits) or sigmoid(logits); experts are picked by score + bias
  (a bias for balance, which has no part in the weights), first among groups of
  experts where there are groups.  A logit of -inf masks an expert; places left over
  hold id -1 and weight 0.  Weights are the picked scores times `scale`, divided by
  their sum where renormalize.  Backward: the gradient of the logits.
* the experts' products: out_t = sum_j w_tj W_out[e] (silu(g) * u) with
  (g, u) = W_in[e] x_t, e = ids_tj; places with an id below 0 count for nothing.
  Backward: gradients of x, W_in, W_out and w.
* the norm over all gradients of a step, and their clipping: outputs are the
  gradients times max_norm / norm where norm > max_norm, else the gradients.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def _route(T, E, k, dtype, train, **more):
    c = {"op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "train": train, "scoring": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_score": "max", "renormalize": True, "scale": 1.0, "masked": 0.0, "pad": 0}
    c.update(more)
    return c


def _experts(T, E, k, D, F, dtype, train, **more):
    c = {"op": "experts", "T": T, "E": E, "k": k, "D": D, "F": F, "dtype": dtype, "train": train, "skew": 0.5,
         "dropped": 0.0, "poison": False, "pad": 0}
    c.update(more)
    return c


def _clip(tensors, total, dtype, clips, **more):
    c = {"op": "clip", "tensors": tensors, "total": total, "dtype": dtype, "clips": clips, "sizes": 1}
    c.update(more)
    return c


def listed():
    return [
        # serving: one token's experts, where only latency counts
        _route(1, 128, 8, "bf16", False, name="route_one_token"),
        # serving: a long prompt batch, sigmoid scores with a bias for balance and groups of experts
        _route(16384, 256, 8, "f32", False, name="route_groups", scoring="sigmoid", bias=True, groups=8, top_groups=4,
               group_score="top2", scale=2.5),
        # training: an odd number of tokens and experts, part of the experts masked, loss gradient back to the logits
        _route(32771, 60, 4, "bf16", True, name="route_train_odd", renormalize=False, masked=0.1),
        # serving: one token through its eight experts
        _experts(1, 64, 8, 2048, 1024, "bf16", False, name="experts_one_token"),
        # serving: a decoding batch that touches nearly every expert
        _experts(64, 128, 8, 2048, 768, "bf16", False, name="experts_decode"),
        # serving: a prefill of 8192 tokens
        _experts(8192, 64, 8, 2048, 1024, "bf16", False, name="experts_prefill"),
        # serving: odd sizes in fp16, rows off every boundary, tokens that no expert takes (never written)
        _experts(1000, 10, 3, 1001, 500, "f16", False, name="experts_odd", dropped=0.2, poison=True, pad=3),
        # training: one step of a large layer with popular and rare experts
        _experts(8192, 32, 4, 2048, 1408, "bf16", True, name="experts_train", skew=1.0, dropped=0.05),
        # training: a short batch in fp16, experts with a handful of rows
        _experts(256, 8, 2, 512, 1024, "f16", True, name="experts_train_small"),
        # training: the gradients of a small model, where launches count
        _clip(30, 200_000, "f32", True, name="clip_small"),
        # training: the gradients of a large layer's experts
        _clip(24, 600_000_000, "bf16", True, name="clip_large"),
        # training: many parameters of odd sizes whose norm is under the limit
        _clip(1000, 20_000_003, "f32", False, name="clip_many"),
    ]


MOST_PRODUCTS = 3 * 8192 * 4 * 2048 * 1408
MOST_WEIGHTS = 64 * 3 * 1024 * 2048


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("route", "route", "experts", "experts", "experts", "clip"))
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        E = groups * log_int(4 if groups > 1 else 8, 256 // groups)
        top_groups = rng.randint(1, groups)
        scoring = rng.choice(("softmax", "sigmoid"))
        return _route(log_int(1, 32768), E, min(log_int(1, 16), E // groups * top_groups), rng.choice(("bf16", "f16", "f32")),
                      rng.random() < 0.5, scoring=scoring, bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                      group_score=rng.choice(("max", "top2")), renormalize=rng.random() < 0.6,
                      scale=rng.choice((1.0, 2.5)), masked=rng.choice((0.0, 0.0, 0.3)), pad=rng.choice((0, 0, 1, 8)))
    if op == "clip":
        dtype = rng.choice(("bf16", "f16", "f32"))
        tensors = log_int(1, 1000)
        return _clip(tensors, tensors * 7 + log_int(1000, 200_000_000), dtype, rng.random() < 0.7, sizes=rng.randint(1, 999))
    train = rng.random() < 0.5
    while True:
        T, E, D, F = log_int(1, 16384), log_int(2, 128), log_int(64, 4096), log_int(64, 4096)
        k = rng.randint(1, min(8, E))
        if rng.random() < 0.7:  # most widths are what programs pick: a multiple of 64
            D, F = max(64, D // 64 * 64), max(64, F // 64 * 64)
        if E * 3 * D * F <= MOST_WEIGHTS and T * k * D * F * (3 if train else 1) <= MOST_PRODUCTS:
            break
    return _experts(T, E, k, D, F, rng.choice(("bf16", "bf16", "f16")), train, skew=rng.choice((0.0, 0.5, 1.5)),
                    dropped=rng.choice((0.0, 0.0, 0.3)), poison=rng.random() < 0.3, pad=rng.choice((0, 0, 1, 8)))


def _sizes(case):
    """Elements of each gradient: from one value to a large share of all, in turn a power of two and an odd number."""
    rng = random.Random(case["sizes"])
    n = case["tensors"]
    parts = [math.exp(rng.uniform(0.0, 6.0)) for _ in range(n)]
    free = case["total"] - n
    sizes = [1 + int(free * p / sum(parts)) for p in parts]
    sizes = [s if i % 2 else max(1, s // 64 * 64) for i, s in enumerate(sizes)]
    sizes[-1] += case["total"] - sum(sizes)
    return sizes


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 29)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, device=dev, generator=gen, dtype=dtype)

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=gen, dtype=torch.float32)

    s = dict(case)
    if case["op"] == "clip":
        # gradients of all sizes beside one another, each with a spread of its own
        sizes = _sizes(case)
        flat = normal(case["total"], dtype=dt) if dt != torch.float16 else normal(case["total"]).to(dt)
        spread = torch.exp(2.0 * normal(len(sizes)) - 4.0).tolist()
        s["grads"] = list(flat.split(sizes))
        for g, f in zip(s["grads"], spread):
            g.mul_(f)
        s["flat"] = torch.empty_like(flat)
        s["outputs"] = list(s["flat"].split(sizes))
        norm = math.sqrt(sum(float(g.float().square().sum(dtype=torch.float64)) for g in s["grads"]))
        s["max_norm"] = norm * (0.3 if case["clips"] else 1.7)
        return s
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        # a router's logits: experts of different popularity, tokens with preferences; rows of a wider product
        wide = normal(T, E + case["pad"]) * 1.5
        wide[:, :E] += 0.5 * normal(E)
        if case["masked"]:
            wide[:, :E].masked_fill_(uniform(T, E) < case["masked"], -math.inf)
            wide[T // 2, :E] = -math.inf  # a token that no expert may take
        s["logits"] = wide.to(dt)[:, :E]
        # as balancing leaves it: against the popular ones, and away from 0
        s["b"] = 0.1 * normal(E) if case["bias"] else None
        if case["train"]:
            s["g"] = normal(T, k)
        return s
    D, F = case["D"], case["F"]
    wide = normal(T, D + case["pad"])
    picks = normal(T, E) + case["skew"] * normal(E)
    ids = torch.topk(picks, k, dim=1).indices
    weights = torch.softmax(torch.gather(picks, 1, ids), dim=1)
    gone = uniform(T) < case["dropped"]
    ids[gone] = -1
    if case["poison"]:
        wide[gone] = float("nan")
    s["x"] = wide.to(dt)[:, :D]
    s["ids"], s["w"] = ids, weights
    s["w_in"] = normal(E, 2 * F, D, dtype=dt) * (1.0 / math.sqrt(D))
    s["w_out"] = normal(E, D, F, dtype=dt) * (1.0 / math.sqrt(F))
    if case["train"]:
        # the gradient that the layers above send back (fp16 programs scale their loss)
        s["g"] = (normal(T, D) * 0.05).to(dt)
    return s


def run(s):
    if s["op"] == "route":
        return _route_own(s) if own else _route_plain(s)
    if s["op"] == "experts":
        return _experts_own(s) if own else _experts_plain(s)
    return _clip_own(s) if own else _clip_plain(s)


# ------------------------------------------------------- the framework's calls

def _route_own(s):
    import tiled_dense_gemm_02_gb300 as tg
    ids, weights = tg.route_experts(s["logits"], s["k"], scoring=s["scoring"], bias=s["b"], groups=s["groups"],
                                    top_groups=s["top_groups"], group_score=s["group_score"],
                                    renormalize=s["renormalize"], scale=s["scale"])
    if not s["train"]:
        return {"ids": ids, "weights": weights}
    d_logits = tg.route_experts_backward(s["logits"], ids, s["g"], scoring=s["scoring"], renormalize=s["renormalize"],
                                         scale=s["scale"])
    return {"ids": ids, "weights": weights, "d_logits": d_logits}


def _experts_own(s):
    import tiled_dense_gemm_02_gb300 as tg
    out, saved = tg.expert_mlp(s["x"], s["w_in"], s["w_out"], s["ids"], s["w"], save=s["train"])
    if not s["train"]:
        return {"out": out}
    dx, dw_in, dw_out, dw = tg.expert_mlp_backward(s["x"], s["w_in"], s["w_out"], s["ids"], s["w"], saved, s["g"])
    return {"out": out, "dx": dx, "dw_in": dw_in, "dw_out": dw_out, "dw": dw}


def _clip_own(s):
    import tiled_dense_gemm_02_gb300 as tg
    norm = tg.clip_gradients(s["grads"], s["max_norm"], outputs=s["outputs"])
    return {"norm": norm, "clipped": s["flat"]}


# ------------------------------------------------------------- the plain form

def _route_plain(s):
    """In 64 bits: picks are whole numbers, and scores next to one another decide them."""
    x = s["logits"].double()
    T, E = x.shape
    there = x > -math.inf
    none = torch.zeros((), dtype=x.dtype, device=x.device)
    low = torch.full((), -math.inf, dtype=x.dtype, device=x.device)
    if s["scoring"] == "softmax":
        top = x.amax(dim=1, keepdim=True)
        e = torch.exp(x - torch.where(top > low, top, none))
        total = e.sum(dim=1, keepdim=True)
        score = e / torch.where(total > 0, total, torch.ones_like(total))
    else:
        score = 1 / (1 + torch.exp(-x))
    key = torch.where(there, score + s["b"].double() if s["b"] is not None else score, low)
    if s["groups"] > 1:
        members = key.view(T, s["groups"], -1)
        best = torch.sort(members, dim=2, descending=True).values[:, :, :1 if s["group_score"] == "max" else 2]
        value = torch.where(best[:, :, 0] > low, torch.where(best > low, best, none).sum(dim=2), low)
        order = torch.sort(value, dim=1, descending=True, stable=True).indices
        rank = torch.argsort(order, dim=1)
        key = torch.where((rank < s["top_groups"])[:, :, None], members, low).reshape(T, E)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :s["k"]]
    used = torch.gather(key, 1, ids) > low
    p = torch.where(used, torch.gather(score, 1, ids), none)
    total = p.sum(dim=1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    w = p / total * s["scale"] if s["renormalize"] else p * s["scale"]
    out = {"ids": torch.where(used, ids, torch.full_like(ids, -1)), "weights": w.float()}
    if s["train"]:
        g = torch.where(used, s["g"].double(), none) * s["scale"]
        if s["renormalize"]:  # to the gradient of the picked scores
            g = torch.where(used, (g - (g * p / total).sum(dim=1, keepdim=True)) / total, none)
        d_score = torch.zeros_like(score).scatter_add_(1, ids, g)
        if s["scoring"] == "softmax":
            d = score * (d_score - (d_score * score).sum(dim=1, keepdim=True))
        else:
            d = d_score * score * (1 - score)
        out["d_logits"] = d.to(s["logits"].dtype)
    return out


def _experts_plain(s):
    T, D = s["x"].shape
    E, k = s["w_in"].shape[0], s["k"]
    F = s["w_out"].shape[2]
    ids, used = s["ids"].reshape(-1), s["ids"].reshape(-1) >= 0
    w = torch.where(used, s["w"].reshape(-1), torch.zeros((), device=ids.device))
    x = torch.where(used.view(T, k).any(dim=1)[:, None], s["x"].float(), torch.zeros((), device=ids.device))
    if not s["train"] and T * k <= E:  # a few rows: each with its expert's weights
        e = torch.where(used, ids, torch.zeros_like(ids))
        gu = torch.matmul(s["w_in"][e].float(), x.repeat_interleave(k, dim=0)[:, :, None])[:, :, 0]
        h = gu[:, :F] / (1 + torch.exp(-gu[:, :F])) * gu[:, F:]
        y = torch.matmul(s["w_out"][e].float(), h[:, :, None])[:, :, 0]
        return {"out": (y * w[:, None]).view(T, k, D).sum(dim=1).to(s["x"].dtype)}
    # rows in their experts' order, each expert's padded to the longest list
    key = torch.where(used, ids, torch.full_like(ids, E))
    order = torch.argsort(key, stable=True)
    count = torch.zeros(E + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    first = torch.cumsum(count, dim=0) - count
    C = max(1, int(count[:E].max()))
    place = torch.arange(T * k, device=ids.device) - first[key[order]]
    # place of every row in the padded lists; what no expert takes goes to a list of its own, which is left out
    at = torch.where(key[order] < E, key[order] * C + place, torch.full_like(place, E * C))
    row = torch.full((E * C + 1,), T, dtype=torch.long, device=ids.device).scatter_(0, at, order // k)[:-1]
    spot = torch.empty_like(at).scatter_(0, order, at)

    def padded(v):
        return torch.cat([v, v.new_zeros(1, v.shape[1])])[row].view(E, C, -1)

    def rows(v):
        return torch.cat([v.reshape(E * C, -1), v.new_zeros(1, v.shape[-1])])[spot]

    w_in, w_out = s["w_in"].float(), s["w_out"].float()
    xp = padded(x)
    gu = torch.bmm(xp, w_in.transpose(1, 2))
    g, u = gu[:, :, :F], gu[:, :, F:]
    sig = 1 / (1 + torch.exp(-g))
    h = g * sig * u
    y = rows(torch.bmm(h, w_out.transpose(1, 2)))
    out = {"out": (y * w[:, None]).view(T, k, D).sum(dim=1).to(s["x"].dtype)}
    if not s["train"]:
        return out
    wp = torch.cat([w.new_zeros(E * C + 1)]).scatter_(0, spot, w)[:-1].view(E, C, 1)
    gp = padded(torch.where(used.view(T, k).any(dim=1)[:, None], s["g"].float(), torch.zeros((), device=ids.device)))
    dh = torch.bmm(gp, w_out)
    out["dw"] = torch.where(used, rows((dh * h).sum(dim=2, keepdim=True))[:, 0], torch.zeros_like(w)).view(T, k)
    out["dw_out"] = torch.bmm((gp * wp).transpose(1, 2), h).to(s["w_out"].dtype)
    dh = dh * wp
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], dim=2)
    out["dw_in"] = torch.bmm(dgu.transpose(1, 2), xp).to(s["w_in"].dtype)
    out["dx"] = rows(torch.bmm(dgu, w_in)).view(T, k, D).sum(dim=1).to(s["x"].dtype)
    return out


def _clip_plain(s):
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]])
    norm = squares.sum().sqrt()
    factor = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm)).float()
    clipped = torch.cat([(g.float() * factor).to(g.dtype) for g in s["grads"]])
    return {"norm": norm.float(), "clipped": clipped}


# --------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _route_exact(s)
    if case["op"] == "experts":
        # 64-bit products run at about 1 TFLOP/s
        return None if work(case)["flops"] > 1.2e13 else _experts_exact(s)
    total = math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"])
    norm = math.sqrt(total)
    factor = min(1.0, s["max_norm"] / norm) if norm else 1.0
    return {"norm": torch.tensor(norm, dtype=torch.float64), "clipped": torch.cat(s["grads"]).double() * factor}


def _route_exact(s):
    logits = s["logits"].double().detach().clone().requires_grad_(s["train"])
    masked = torch.isneginf(logits)
    if s["scoring"] == "softmax":
        log_score = logits - torch.logsumexp(logits, dim=1, keepdim=True)
        log_score = torch.where(masked, torch.full_like(log_score, -math.inf), log_score)
    else:
        log_score = torch.nn.functional.logsigmoid(logits)
    T, E = logits.shape
    free = torch.where(masked, torch.full_like(logits, -math.inf), torch.exp(log_score.detach()))
    if s["b"] is not None:
        free = free + s["b"].double()
    if s["groups"] > 1:
        size = E // s["groups"]
        value = torch.full((T, s["groups"]), -math.inf, dtype=torch.float64, device=logits.device)
        for i in range(s["groups"]):
            part = free[:, i * size:(i + 1) * size]
            top = part.amax(dim=1)
            value[:, i] = top
            if s["group_score"] == "top2" and size > 1:
                rest = part.scatter(1, part.argmax(dim=1, keepdim=True), -math.inf).amax(dim=1)
                value[:, i] = torch.where(rest > -math.inf, top + rest, top)
        keep = torch.zeros_like(value, dtype=torch.bool)
        for _ in range(s["top_groups"]):
            keep.scatter_(1, _first_largest(value)[:, None], True)
            value = value.masked_fill(keep, -math.inf)
        free = free.masked_fill(~keep.repeat_interleave(size, dim=1), -math.inf)
    ids = []
    for _ in range(s["k"]):
        best = _first_largest(free)
        ids.append(torch.where(free.amax(dim=1) > -math.inf, best, torch.full_like(best, -1)))
        free = free.scatter(1, best[:, None], -math.inf)
    ids = torch.stack(ids, dim=1)
    used = ids >= 0
    picked = torch.gather(log_score, 1, ids.clamp_min(0))
    picked = torch.where(used, picked, torch.full_like(picked, -math.inf))
    if s["renormalize"]:
        total = torch.logsumexp(torch.where(used.any(dim=1, keepdim=True), picked, torch.zeros_like(picked)), dim=1, keepdim=True)
        picked = picked - total
    w = torch.where(used, torch.exp(torch.where(used, picked, torch.zeros_like(picked))), torch.zeros_like(picked)) * s["scale"]
    out = {"ids": ids, "weights": w.detach()}
    if s["train"]:
        # by differences of the logarithm: a weight's gradient with respect to the picked scores' logarithms, then to the logits
        g = torch.where(used, s["g"].double(), torch.zeros_like(w)) * w.detach()
        if s["renormalize"]:
            g = g - w.detach() / s["scale"] * g.sum(dim=1, keepdim=True)
        score = torch.where(masked, torch.zeros_like(logits), torch.exp(log_score)).detach()
        spread = torch.zeros_like(score).scatter_add_(1, ids.clamp_min(0), g)
        out["d_logits"] = spread - score * g.sum(dim=1, keepdim=True) if s["scoring"] == "softmax" else spread * (1 - score)
    return out


def _first_largest(v):
    """Index of each row's largest value, the lowest one of several."""
    at = torch.arange(v.shape[1], device=v.device).expand_as(v)
    return torch.where(v == v.amax(dim=1, keepdim=True), at, torch.full_like(at, v.shape[1])).amin(dim=1).clamp_max(v.shape[1] - 1)


def _experts_exact(s):
    T, D = s["x"].shape
    E, F = s["w_in"].shape[0], s["w_out"].shape[2]
    f64 = {"dtype": torch.float64, "device": s["x"].device}
    out = {"out": torch.zeros(T, D, **f64)}
    if s["train"]:
        out |= {"dx": torch.zeros(T, D, **f64), "dw_in": torch.zeros(E, 2 * F, D, **f64),
                "dw_out": torch.zeros(E, D, F, **f64), "dw": torch.zeros(T, s["k"], **f64)}
    for e in range(E):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if not t.numel():
            continue
        x, a, b = s["x"][t].double(), s["w_in"][e].double(), s["w_out"][e].double()
        w = s["w"][t, j].double()[:, None]
        g, u = x @ a[:F].t(), x @ a[F:].t()
        h = torch.nn.functional.silu(g) * u
        out["out"].index_add_(0, t, w * (h @ b.t()))
        if s["train"]:
            up = s["g"][t].double()
            out["dw"][t, j] = (up * (h @ b.t())).sum(dim=1)
            out["dw_out"][e] = (w * up).t() @ h
            dh = (w * up) @ b
            sig = torch.sigmoid(g)
            dg, du = dh * u * (sig + g * sig * (1 - sig)), dh * torch.nn.functional.silu(g)
            out["dw_in"][e, :F], out["dw_in"][e, F:] = dg.t() @ x, du.t() @ x
            out["dx"].index_add_(0, t, dg @ a[:F] + du @ a[F:])
    return out


def work(case):
    """Inputs read once, outputs written once.  A forward pass of the experts reads the weights of those that its rows
    touch (on average); a training step writes every expert's gradients."""
    es = BYTES[case["dtype"]]
    if case["op"] == "clip":
        return {"bytes": 2.0 * es * case["total"] + 4, "flops": 3.0 * case["total"]}
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        b, f = T * E * es + T * k * 12, 8.0 * T * E
        return {"bytes": float(b + T * k * 12 + 2 * T * E * es if case["train"] else b), "flops": 2 * f if case["train"] else f}
    D, F = case["D"], case["F"]
    rows = max(1.0, T * k * (1.0 - case["dropped"]))
    touched = E * (1.0 - (1.0 - 1.0 / E) ** rows)
    lists = T * k * 12
    if case["train"]:
        b = 4 * T * D * es + (touched + E) * 3 * D * F * es + lists + 4 * T * k
        return {"bytes": float(b), "flops": 18.0 * rows * D * F}
    return {"bytes": float(2 * T * D * es + touched * 3 * D * F * es + lists), "flops": 6.0 * rows * D * F}
