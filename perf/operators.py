"""The vocabulary-head losses: what is measured of them, and their plain form.

Two operators, each with its backward pass, work on hidden states H [T, D] and the
head's weight W [V, D] (one row per vocabulary entry) without ever holding the
T x V logits z = scale * H W^T:

* linear cross entropy: with q = (1 - eps) 1[v = target] + eps / V,
  loss_t = lse_t - sum_v q_v z_tv + z_loss * lse_t^2,   lse_t = log sum_v exp(z_tv);
* linear distillation: with q = softmax of the teacher's K listed logits / tau and
  z = H W^T / tau, loss_t = sum_k q_k log q_k + lse_t - sum_k q_k z_t,id_k.

Backward, with g the gradient of the losses: dz = g ((1 + 2 z_loss lse) softmax(z) - q),
dH = scale * dz W, dW = scale * dz^T H.  Rows whose target is the ignored index, or
whose teacher lists nothing, have loss, lse and gradients 0, whatever H holds there.
"""
import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def _case(op, T, V, D, dtype, train, **more):
    c = {"op": op, "T": T, "V": V, "D": D, "dtype": dtype, "train": train, "ignored": 0.0, "pad": 0, "poison": False,
         "weighted": False, "smoothing": 0.0, "z_loss": 0.0, "scale": 1.0, "K": 0}
    c.update(more)
    return c


def listed():
    return [
        # serving: the log-probability of one sampled token
        _case("xent", 1, 32768, 4096, "bf16", False, name="score_one_token"),
        # serving: a short batch scored under an odd vocabulary and an odd hidden width, rows off every boundary
        _case("xent", 77, 50021, 1001, "f16", False, name="score_batch_odd", ignored=0.1),
        # evaluation: the perplexity of one 2048-token window over a large vocabulary
        _case("xent", 2048, 131072, 4096, "bf16", False, name="evaluate_window"),
        # pre-training: one step's head on 8192 tokens, loss and both gradients
        _case("xent", 8192, 131072, 4096, "bf16", True, name="train_large", ignored=0.05),
        # instruction tuning: prompts and padding (never written) are ignored; weighted tokens, smoothing, z-loss,
        # hidden states that are a slice of wider rows
        _case("xent", 4096, 65536, 2048, "bf16", True, name="train_masked", ignored=0.6, pad=64, poison=True,
              weighted=True, smoothing=0.1, z_loss=1e-4),
        # fine-tuning of a small head on a short batch in fp16
        _case("xent", 128, 32768, 1024, "f16", True, name="train_small", scale=0.5),
        # a small model trained in fp32
        _case("xent", 512, 16384, 512, "f32", True, name="train_f32", ignored=0.1),
        # checking a student against stored teacher logits, a few tokens at a time
        _case("distill", 64, 131072, 2048, "bf16", False, name="distill_check", K=64, scale=0.5),
        # distillation step on 4096 tokens, 64 stored teacher logits per token
        _case("distill", 4096, 131072, 2048, "bf16", True, name="distill_train", K=64, scale=0.5, ignored=0.05),
        # distillation at odd sizes in fp16: rows off the 16-byte grid, lists of different lengths
        _case("distill", 1000, 50021, 1500, "f16", True, name="distill_ragged", K=17, ignored=0.3, weighted=True,
              scale=0.25),
        # a handful of tokens and a short list: latency of a training step
        _case("distill", 33, 8192, 512, "bf16", True, name="distill_few", K=8, scale=1.0),
        # distillation in fp32
        _case("distill", 256, 8192, 1024, "f32", True, name="distill_f32", K=32, scale=0.5, ignored=0.1),
    ]


MOST_WORK = 8192 * 131072 * 4096


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("xent", "distill"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f16", "f32"))
    train = rng.random() < 0.6
    most = MOST_WORK // (64 if dtype == "f32" else 2)
    while True:
        T, V, D = log_int(1, 8192), log_int(1000, 131072), log_int(64, 4096)
        if rng.random() < 0.5:  # half of the sizes are what programs pick: a multiple of 64
            D, V = max(64, D // 64 * 64), max(1024, V // 64 * 64)
        if T * V * D <= most:
            break
    c = _case(op, T, V, D, dtype, train, ignored=rng.choice((0.0, 0.1, 0.5)), pad=rng.choice((0, 0, 1, 8)),
              poison=rng.random() < 0.3, weighted=rng.random() < 0.5, scale=rng.choice((1.0, 0.5, 0.25)))
    if op == "distill":
        c["K"] = log_int(1, 128)
    elif rng.random() < 0.5:
        c["smoothing"], c["z_loss"] = 0.1, 1e-4
    return c


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 17)
    T, V, D, dt = case["T"], case["V"], case["D"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=gen, dtype=torch.float32)

    # a trained head: rows of norm about 2, so that logits / scale spread with a deviation of about 2
    w = torch.empty(V, D, device=dev, dtype=dt)
    for lo in range(0, V, 16384):
        n = min(V, lo + 16384) - lo
        w[lo:lo + n] = (normal(n, D) * (2.0 / math.sqrt(D))).to(dt)
    # tokens as frequent as in text (a power law over the vocabulary), and hidden states that know something of them
    target = (torch.exp(uniform(T) * math.log(V)) - 1).long().clamp_(0, V - 1)
    wide = normal(T, D + case["pad"])
    wide[:, :D] += w[target].float() * (2.0 * uniform(T, 1))
    dropped = uniform(T) < case["ignored"]
    if case["poison"]:
        wide[dropped] = float("nan")
    h = wide.to(dt)[:, :D]
    s = {"op": case["op"], "train": case["train"], "h": h, "w": w, "scale": case["scale"],
         "smoothing": case["smoothing"], "z_loss": case["z_loss"]}
    if case["op"] == "xent":
        s["target"] = torch.where(dropped, torch.full_like(target, IGNORE), target)
    else:
        K = min(case["K"], V)
        # K distinct entries a row, the token itself first; logits that fall off as a teacher's do
        step = 1 + (uniform(T, 1) * max(1, V // K - 1)).long()
        rank = torch.argsort(uniform(T, K), dim=1) if K > 1 else torch.zeros(T, 1, dtype=torch.long, device=dev)
        rank[:, 1:] = torch.where(rank[:, 1:] == 0, rank[:, :1].expand(-1, K - 1), rank[:, 1:])
        rank[:, 0] = 0
        ids = (target[:, None] + rank * step) % V
        logits = 12.0 - 2.0 * torch.log1p(torch.arange(K, device=dev, dtype=torch.float32)) + 0.5 * normal(T, K)
        # shorter lists in part of the rows, and rows whose list is empty
        length = torch.where(uniform(T) < 0.25, (1 + uniform(T) * K).long().clamp_(max=K), torch.full_like(target, K))
        length = torch.where(dropped, torch.zeros_like(length), length)
        s["ids"] = torch.where(torch.arange(K, device=dev)[None, :] < length[:, None], ids, torch.full_like(ids, -1))
        s["logits"] = logits
    if case["train"]:
        # the gradient of the mean over the tokens that count, or of a weighted mean
        g = torch.where(dropped, torch.zeros(T, device=dev), torch.ones(T, device=dev))
        g = g * (0.25 + uniform(T)) if case["weighted"] else g
        s["g"] = g / max(1.0, float((~dropped).sum()))
    return s


def run(s):
    if own:
        import tiled_dense_gemm_02_gb300 as tg
        if s["op"] == "xent":
            more = {"ignore_index": IGNORE, "scale": s["scale"], "label_smoothing": s["smoothing"], "z_loss": s["z_loss"]}
            loss, lse = tg.linear_cross_entropy(s["h"], s["w"], s["target"], **more)
            if s["train"]:
                dh, dw = tg.linear_cross_entropy_backward(s["h"], s["w"], s["target"], lse, s["g"], **more)
        else:
            more = {"temperature": 1.0 / s["scale"]}
            loss, lse = tg.linear_distillation(s["h"], s["w"], s["ids"], s["logits"], **more)
            if s["train"]:
                dh, dw = tg.linear_distillation_backward(s["h"], s["w"], s["ids"], s["logits"], lse, s["g"], **more)
    elif s["op"] == "xent":
        loss, lse, dh, dw = _plain_xent(s)
    else:
        loss, lse, dh, dw = _plain_distill(s)
    return {"loss": loss, "lse": lse, "dh": dh, "dw": dw} if s["train"] else {"loss": loss, "lse": lse}


# ------------------------------------------------------------- the plain form

def _plain_logits(s, counts):
    h = torch.where(counts[:, None], s["h"].float(), torch.zeros((), device=s["h"].device))
    w = s["w"].float()
    z = (h @ w.t()) * s["scale"]
    top = z.amax(dim=1, keepdim=True)
    lse = (z - top).exp().sum(dim=1).log() + top[:, 0]
    return h, w, z, lse


def _plain_gradients(s, h, w, dz):
    dh = (dz @ w) * s["scale"]
    dw = (dz.t() @ h) * s["scale"]
    return dh.to(s["h"].dtype), dw.to(s["w"].dtype)


def _plain_xent(s):
    counts = s["target"] != IGNORE
    at = torch.where(counts, s["target"], torch.zeros_like(s["target"]))[:, None]
    h, w, z, lse = _plain_logits(s, counts)
    V, eps = w.shape[0], s["smoothing"]
    loss = lse - (1 - eps) * z.gather(1, at)[:, 0] + s["z_loss"] * lse * lse
    if eps:
        loss = loss - eps * (z.sum(dim=1) / V)
    zero = torch.zeros_like(lse)
    out, out_lse = torch.where(counts, loss, zero), torch.where(counts, lse, zero)
    if not s["train"]:
        return out, out_lse, None, None
    g = torch.where(counts, s["g"], zero)[:, None]
    dz = z.sub_(lse[:, None]).exp_().mul_(1 + 2 * s["z_loss"] * lse[:, None]).sub_(eps / V)
    dz.scatter_add_(1, at, torch.full_like(at, -(1 - eps), dtype=dz.dtype))
    return (out, out_lse) + _plain_gradients(s, h, w, dz.mul_(g))


def _plain_distill(s):
    there = s["ids"] >= 0
    counts = there.any(dim=1)
    at = torch.where(there, s["ids"], torch.zeros_like(s["ids"]))
    h, w, z, lse = _plain_logits(s, counts)
    t = torch.where(there, s["logits"] * s["scale"], torch.full_like(s["logits"], -3e38))
    e = torch.where(there, (t - t.amax(dim=1, keepdim=True)).exp(), torch.zeros_like(t))
    total = e.sum(dim=1, keepdim=True)
    q = e / torch.where(counts[:, None], total, torch.ones_like(total))
    own_term = torch.where(q > 0, q * torch.where(q > 0, q, torch.ones_like(q)).log(), torch.zeros_like(q)).sum(dim=1)
    loss = own_term + lse - (q * z.gather(1, at)).sum(dim=1)
    zero = torch.zeros_like(lse)
    out, out_lse = torch.where(counts, loss, zero), torch.where(counts, lse, zero)
    if not s["train"]:
        return out, out_lse, None, None
    g = torch.where(counts, s["g"], zero)[:, None]
    dz = z.sub_(lse[:, None]).exp_()
    dz.scatter_add_(1, at, -q)
    return (out, out_lse) + _plain_gradients(s, h, w, dz.mul_(g))


# --------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    T, V, D = case["T"], case["V"], case["D"]
    kept = torch.nonzero(s["target"] != IGNORE if case["op"] == "xent" else (s["ids"] >= 0).any(dim=1))[:, 0]
    n, one = int(kept.numel()), 2.0 * T * V * D
    if one > 1.2e13:
        return None
    # the gradients of the largest cases would take minutes in 64 bits
    grads = case["train"] and 3 * one <= 1.2e13
    dev = s["h"].device
    h = s["h"][kept].double()
    step = max(1, min(V, (1 << 28) // max(1, n)))
    pieces = [(lo, min(V, lo + step)) for lo in range(0, V, step)]
    # the distribution q of every kept row as a list of entries and masses
    if case["op"] == "xent":
        ids = s["target"][kept][:, None]
        mass = torch.full((n, 1), 1.0 - case["smoothing"], dtype=torch.float64, device=dev)
        own_term = torch.zeros(n, dtype=torch.float64, device=dev)
    else:
        ids = s["ids"][kept]
        t = (s["logits"][kept].double() * case["scale"]).masked_fill(ids < 0, -math.inf)
        logq = torch.log_softmax(t, dim=1)
        mass = logq.exp()
        own_term = torch.special.xlogy(mass, mass).sum(dim=1)
    flat = case["smoothing"] / V if case["op"] == "xent" else 0.0
    zl = case["z_loss"] if case["op"] == "xent" else 0.0
    lse = torch.full((n,), -math.inf, dtype=torch.float64, device=dev)
    dot = torch.zeros(n, dtype=torch.float64, device=dev)

    def piece(lo, hi):
        w = s["w"][lo:hi].double()
        inside = (ids >= lo) & (ids < hi)
        return w, torch.mm(h, w.t()) * case["scale"], inside, torch.where(inside, ids - lo, torch.zeros_like(ids))

    for lo, hi in pieces:
        w, z, inside, at = piece(lo, hi)
        lse = torch.logaddexp(lse, torch.logsumexp(z, dim=1))
        dot += torch.where(inside, mass * torch.gather(z, 1, at), torch.zeros_like(mass)).sum(dim=1)
        if flat:
            dot += flat * z.sum(dim=1)
    out = {"loss": torch.zeros(T, dtype=torch.float64, device=dev), "lse": torch.zeros(T, dtype=torch.float64, device=dev)}
    out["loss"][kept] = own_term + lse - dot + zl * lse * lse
    out["lse"][kept] = lse
    if case["train"]:
        out["dh"] = out["dw"] = None
    if grads:
        g = s["g"][kept].double()
        dh = torch.zeros(n, D, dtype=torch.float64, device=dev)
        dw = torch.zeros(V, D, dtype=torch.float64, device=dev)
        for lo, hi in pieces:
            w, z, inside, at = piece(lo, hi)
            dz = torch.exp(z - lse[:, None]) * (1 + 2 * zl * lse)[:, None] - flat
            dz.scatter_add_(1, at, -torch.where(inside, mass, torch.zeros_like(mass)))
            dz *= (g * case["scale"])[:, None]
            dh += torch.mm(dz, w)
            dw[lo:hi] = torch.mm(dz.t(), h)
        out["dh"] = torch.zeros(T, D, dtype=torch.float64, device=dev)
        out["dh"][kept] = dh
        out["dw"] = dw
    return out


def work(case):
    """Inputs read once, outputs written once; one product for the logits and, in training, two for the gradients,
    over the rows that count (on average)."""
    T, V, D, K = case["T"], case["V"], case["D"], case["K"]
    e = BYTES[case["dtype"]]
    rows = max(1.0, T * (1.0 - case["ignored"]))
    matrices = (rows * D + V * D) * e
    lists = T * 8 if case["op"] == "xent" else T * K * 12
    flops = 2.0 * rows * V * D
    if case["train"]:
        return {"bytes": 2 * matrices + lists + 3 * 4 * T, "flops": 3 * flops}
    return {"bytes": matrices + lists + 2 * 4 * T, "flops": flops}
