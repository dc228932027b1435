"""What is measured of the loss and clipping operators.

Each case is one pass through one operator: token log-probabilities (`logprob`),
the clipped policy loss with its KL term (`policy`), the preference loss over
pairs (`preference`), and the global norm with clipping (`clip`).  Where `own`
is false, `run` computes the operator in elementary torch operations in 32
bits; where it is true, it calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of one request: score the token that was drawn (latency)
        {"name": "logprob decode", "op": "logprob", "rows": 1, "vocab": 131072, "dtype": "bf16", "entropy": False,
         "backward": False, "temperature": 1.0, "ignored": 0.0},
        # scoring a batch under the reference policy; a vocabulary of odd size puts every row on another alignment
        {"name": "logprob scoring", "op": "logprob", "rows": 4099, "vocab": 50001, "dtype": "f16", "entropy": False,
         "backward": False, "temperature": 1.0, "ignored": 0.0},
        # a loss of the user's own on log-probabilities and entropies: forward, then the gradient of the logits
        {"name": "logprob training", "op": "logprob", "rows": 6000, "vocab": 32000, "dtype": "bf16", "entropy": True,
         "backward": True, "temperature": 0.7, "ignored": 0.1},
        # an actor's head over a few actions, some of them not allowed (-inf), with the entropy bonus (latency)
        {"name": "policy actions", "op": "policy", "rows": 256, "vocab": 18, "dtype": "f32", "entropy": True, "kl": False,
         "sequences": 0, "temperature": 1.0, "masked": 0.3, "ignored": 0.0},
        # one micro-batch of a token policy, one advantage to a sequence, mean over counted tokens, prompts ignored
        {"name": "policy micro-batch", "op": "policy", "rows": 2048, "vocab": 32768, "dtype": "bf16", "entropy": False, "kl": True,
         "sequences": 8, "temperature": 1.0, "masked": 0.0, "ignored": 0.2},
        # a whole batch over a large vocabulary: offsets past 2^31 elements
        {"name": "policy batch", "op": "policy", "rows": 16391, "vocab": 131072, "dtype": "bf16", "entropy": False, "kl": True,
         "sequences": 16, "temperature": 1.0, "masked": 0.0, "ignored": 0.1},
        # a few short pairs over a small output layer in 32 bits (latency)
        {"name": "preference short", "op": "preference", "rows": 97, "pairs": 2, "vocab": 1000, "dtype": "f32", "kind": "sigmoid",
         "average": False, "ignored": 0.0},
        # ragged pairs, odd vocabulary, length-normalised squared loss
        {"name": "preference odd", "op": "preference", "rows": 3001, "pairs": 4, "vocab": 50001, "dtype": "bf16", "kind": "ipo",
         "average": True, "ignored": 0.2},
        # a batch of long pairs over a large vocabulary
        {"name": "preference batch", "op": "preference", "rows": 12000, "pairs": 12, "vocab": 128000, "dtype": "bf16", "kind": "sigmoid",
         "average": False, "ignored": 0.3},
        # a small fully connected net's gradients (latency)
        {"name": "clip small", "op": "clip", "set": "mlp", "width": 96, "count": 6, "dtype": "f32", "metric": False, "step": False},
        # ResNet-50's tensors: natural gradient steps bounded in the curvature's metric, and the step on the weights
        {"name": "clip resnet50 step", "op": "clip", "set": "resnet50", "width": 0, "count": 161, "dtype": "f32", "metric": True, "step": True},
        # a large model's 16-bit gradients
        {"name": "clip large", "op": "clip", "set": "blocks", "width": 4096, "count": 48, "dtype": "bf16", "metric": False, "step": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprob", "policy", "preference", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "clip":
        kind = rng.choice(["mlp", "blocks"])
        width = _log(rng, 16, 4096)
        most = max(2, min(300, 1_600_000_000 // (width * width * 2 * SIZE[dtype])))
        metric = rng.random() < 0.5
        return {"op": op, "set": kind, "width": width, "count": rng.randint(1, most), "dtype": dtype, "metric": metric,
                "step": rng.random() < 0.5}
    vocab = _log(rng, 4, 200_000)
    top = max(2, min(20_000, 1_000_000_000 // vocab * 2 // SIZE[dtype]))
    rows = _log(rng, 1 if op == "logprob" else 4, max(top, 5))
    if op == "logprob":
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "entropy": rng.random() < 0.5, "backward": rng.random() < 0.6,
                "temperature": rng.choice([1.0, 0.7, 1.3]), "ignored": rng.choice([0.0, 0.2])}
    if op == "policy":
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "entropy": rng.random() < 0.5, "kl": rng.random() < 0.6,
                "sequences": rng.choice([0, rng.randint(1, max(1, min(64, rows // 4)))]), "temperature": rng.choice([1.0, 0.8]),
                "masked": rng.choice([0.0, 0.3]), "ignored": rng.choice([0.0, 0.2])}
    pairs = rng.randint(max(1, rows // 2000), max(1, min(64, rows // 4)))
    return {"op": op, "rows": rows, "pairs": pairs, "vocab": vocab, "dtype": dtype,
            "kind": rng.choice(["sigmoid", "hinge", "ipo"]), "average": rng.random() < 0.5, "ignored": rng.choice([0.0, 0.2])}


def _shapes(case):
    """The gradients' shapes of a clip case."""
    n, w = case["count"], case["width"]
    if case["set"] == "mlp":  # layers with bias vectors
        return [(w, w + 1) if k % 2 == 0 else (w,) for k in range(n)]
    if case["set"] == "blocks":  # square, wide and tall matrices, and the norms' vectors
        return [[(w, w), (w, 2 * w), (2 * w, w), (w + 1,)][k % 4] for k in range(n)]
    out, cin = [(64, 147), (64,), (64,)], 64
    for blocks, width, cout in ((3, 64, 256), (4, 128, 512), (6, 256, 1024), (3, 512, 2048)):
        for b in range(blocks):
            convs = [(width, cin), (width, 9 * width), (cout, width)] + ([(cout, cin)] if b == 0 else [])
            out += [s for c in convs for s in (c, (c[0],), (c[0],))]
            cin = cout
    return out + [(1000, 2048), (1000,)]


def work(case):
    """Bytes that each input is read and each output written once, and the
    operations on each element."""
    e = SIZE[case["dtype"]]
    if case["op"] == "clip":
        n = sum(math.prod(s) for s in _shapes(case))
        reads = e * (2 if case["metric"] else 1) + (4 if case["step"] else 0)
        return {"bytes": n * (reads + (4 if case["step"] else e)), "flops": n * (5 if case["step"] else 3)}
    n, r = case["rows"] * case["vocab"], case["rows"]
    read = int(n * (1 - case["ignored"])) * e  # an ignored row is not read, its gradient is zeros
    if case["op"] == "logprob":
        return {"bytes": read + (n * e if case["backward"] else 0) + r * 24, "flops": n * (8 if case["backward"] else 4)}
    return {"bytes": read + n * e + r * 32, "flops": n * 8}


# ------------------------------------------------------------------ the inputs

def _logits(case, gen):
    """Logits as a language model's are: a few frequent tokens far above a long tail."""
    rows, vocab, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    bias = -2.0 * torch.log(torch.arange(1, vocab + 1, device="cuda", dtype=torch.float32))
    bias = (bias - bias.mean())[torch.randperm(vocab, device="cuda", generator=gen)]
    z = torch.empty(rows, vocab, dtype=dt, device="cuda")
    target = torch.empty(rows, dtype=torch.int64, device="cuda")
    lse = torch.empty(rows, device="cuda")
    tau = case.get("temperature", 1.0)
    step = max(1, (1 << 28) // vocab)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        x = torch.randn(b - a, vocab, device="cuda", generator=gen).mul_(1.5).add_(bias)
        if case.get("masked"):  # actions that are not allowed; the first one always is
            off = torch.rand(b - a, vocab, device="cuda", generator=gen) < case["masked"]
            off[:, 0] = False
            x.masked_fill_(off, -math.inf)
        z[a:b] = x
        x = z[a:b].float() / tau
        lse[a:b] = torch.logsumexp(x, 1)
        x -= torch.empty_like(x).exponential_(generator=gen).log_()  # the token that the policy drew
        target[a:b] = x.argmax(1)
        del x
    logp = z.gather(1, target[:, None])[:, 0].float() / tau - lse
    if case["ignored"]:
        target[torch.rand(rows, device="cuda", generator=gen) < case["ignored"]] = -100
    return z, target, logp


def _offsets(rows, parts, gen):
    """Where `parts` sequences of ragged lengths start, and where the last one ends."""
    share = torch.rand(parts, device="cuda", generator=gen) + 0.3
    ends = (share.cumsum(0) / share.sum() * rows).round().to(torch.int32)
    ends[-1] = rows
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), ends])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    s = {"case": case}
    if case["op"] == "clip":
        shapes, dt = _shapes(case), DTYPES[case["dtype"]]
        sizes = [math.prod(x) for x in shapes]
        at = [sum(sizes[:k]) for k in range(len(sizes))]
        views = lambda flat: [flat[a:a + n].view(x) for a, n, x in zip(at, sizes, shapes)]  # noqa: E731
        scale = [10.0 ** (-2.0 - (k % 3)) for k in range(len(shapes))]  # layers' gradients differ in size
        s["x"] = [(normal(*x) * c).to(dt) for x, c in zip(shapes, scale)]
        if case["metric"]:  # steps and gradients point roughly the same way
            s["y"] = [(v.float() * 0.1 + normal(*v.shape) * (0.05 * c)).to(dt) for v, c in zip(s["x"], scale)]
        total = float(sum((a.double() * b.double()).sum() for a, b in zip(s["x"], s.get("y", s["x"]))))
        s["max_norm"] = 0.4 * math.sqrt(total)  # a step that has to be shortened
        if case["step"]:  # the tensors are parts of one allocation
            s["w_all"] = normal(sum(sizes)) * 0.05
            s["w"] = views(s["w_all"])
            s["eta"] = 0.1
        else:
            s["out_all"] = torch.empty(sum(sizes), dtype=dt, device="cuda")
            s["out"] = views(s["out_all"])
        return s
    s["logits"], s["target"], logp = _logits(case, gen)
    rows = case["rows"]
    if case["op"] == "logprob":
        if case["backward"]:  # the gradients that the user's loss sends back
            s["dlogp"] = normal(rows) / rows
            s["dentropy"] = normal(rows) * (0.1 / rows)
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    s["dlogits"] = torch.empty_like(s["logits"])
    if case["op"] == "policy":
        s["old_logp"] = logp + 0.15 * normal(rows)
        if case["kl"]:
            s["ref_logp"] = logp + 0.3 * normal(rows)
        if case["sequences"]:
            s["offsets"] = _offsets(rows, case["sequences"], gen)
            s["advantage"] = normal(case["sequences"]) + 0.5
        else:
            s["advantage"] = normal(rows) + 0.5
        return s
    s["offsets"] = _offsets(rows, 2 * case["pairs"], gen)
    counted = torch.where(s["target"] >= 0, logp, 0.0)
    sums = torch.cat([torch.zeros(1, device="cuda", dtype=torch.float64), counted.double().cumsum(0)])[s["offsets"].long()].diff()
    if case["average"]:
        n = torch.cat([torch.zeros(1, device="cuda"), (s["target"] >= 0).float().cumsum(0)])[s["offsets"].long()].diff()
        sums = sums / n.clamp(min=1)
    s["ref"] = (sums + normal(2 * case["pairs"]) * (0.2 if case["average"] else 4.0)).float()
    return s


# ------------------------------------------------------------------ the passes

CLIP, KL, ENT, BETA = 0.2, 0.04, 0.01, 0.1


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from second_order_optimisation_gb300 import kfac
    c = s["case"]
    if c["op"] == "clip":
        if "list" not in s:  # a training loop keeps its gradient buffers, and this list of them
            none = [None] * len(s["x"])
            s["list"] = kfac.ClipList([kfac.ClipTensor(x, out, y, w) for x, out, y, w in
                                       zip(s["x"], s.get("out", none), s.get("y", none), s.get("w", none))])
        norm, scale = (torch.empty(1, device="cuda") for _ in range(2))
        kfac.kfac_clip_norm(s["list"], s["max_norm"], norm=norm, scale=scale, eta=s.get("eta", 0.0))
        return {"norm": norm, "scale": scale, "out": s["w_all"] if c["step"] else s["out_all"]}
    rows = c["rows"]
    new = lambda n: torch.empty(n, device="cuda")  # noqa: E731
    if c["op"] == "logprob":
        logp, lse, ent = new(rows), new(rows), new(rows) if c["entropy"] else None
        saved = new(2 * rows) if c["backward"] else None
        kfac.kfac_token_logprob(kfac.TokenLogprob(s["logits"], s["target"], logp, lse, ent, c["temperature"], saved))
        out = {"logp": logp, "lse": lse}
        if c["entropy"]:
            out["entropy"] = ent
        if c["backward"]:
            kfac.kfac_token_logprob_grad(kfac.TokenLogprobGrad(
                s["logits"], s["target"], saved, s["dlogp"], s["dlogits"], ent, s["dentropy"] if c["entropy"] else None, c["temperature"]))
            out["dlogits"] = s["dlogits"]
        return out
    if c["op"] == "policy":
        stats, logp, ent = new(5), new(rows), new(rows) if c["entropy"] else None
        kfac.kfac_policy_loss(kfac.PolicyLoss(
            s["logits"], s["target"], s["advantage"], s["old_logp"], stats, logp, s["dlogits"], ref_logp=s.get("ref_logp"),
            seq_offsets=s.get("offsets"), entropy=ent, clip_low=CLIP, clip_high=CLIP, kl_coef=KL if c["kl"] else 0.0,
            entropy_coef=ENT if c["entropy"] else 0.0, temperature=c["temperature"]))
        out = {"loss": stats[0], "logp": logp, "dlogits": s["dlogits"]}
        if c["entropy"]:
            out["entropy"] = ent
        return out
    loss, pair, logp = new(1), new(c["pairs"]), new(2 * c["pairs"])
    kfac.kfac_preference_loss(kfac.PreferenceLoss(
        s["logits"], s["target"], s["offsets"], loss, logp, s["dlogits"], ref_logp=s["ref"], pair_loss=pair,
        kind=c["kind"], beta=BETA, average=c["average"]))
    return {"loss": loss[0], "pair_loss": pair, "logp": logp, "dlogits": s["dlogits"]}


def _softmax(z, target, tau, entropy):
    """p, log p where p > 0 (else 0), the target's log p, lse and the entropy of each row, in 32 bits."""
    x = z.float()
    if tau != 1.0:
        x = x / tau
    m = x.amax(1, keepdim=True)
    x = x - m
    e = torch.exp(x)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    lse = (m + log_total)[:, 0]
    logp = (x.gather(1, target.clamp(min=0)[:, None]) - log_total)[:, 0]
    p = e / total
    lp = h = None
    if entropy:
        lp = torch.where(p > 0, x - log_total, 0.0)
        h = -(p * lp).sum(1)
    return p, lp, logp, lse, h


def _dlogits(s, p, lp, h, g, gh):
    """g (1[j = target] - p) - gh p (lp + h), over the temperature; rows without a target get zeros."""
    live = s["target"] >= 0
    g = torch.where(live, g, 0.0)[:, None]
    d = -g * p
    if gh is not None:
        d = d - torch.where(live, gh, 0.0)[:, None] * p * (lp + h[:, None])
    d.scatter_add_(1, s["target"].clamp(min=0)[:, None], g)
    tau = s["case"].get("temperature", 1.0)
    s["dlogits"].copy_(d / tau if tau != 1.0 else d)
    return s["dlogits"]


def _plain(s):
    c = s["case"]
    if c["op"] == "clip":
        x = s["x"]
        norm = torch.sqrt(torch.stack([(a.float() * b.float()).sum() for a, b in zip(x, s.get("y", x))]).sum()).reshape(1)
        scale = torch.clamp(s["max_norm"] / norm, max=1.0)
        if c["step"]:
            [w.sub_(s["eta"] * (scale * a.float())) for w, a in zip(s["w"], x)]
        else:
            [o.copy_(scale * a.float()) for o, a in zip(s["out"], x)]
        return {"norm": norm, "scale": scale, "out": s["w_all"] if c["step"] else s["out_all"]}
    live = s["target"] >= 0
    p, lp, logp, lse, h = _softmax(s["logits"], s["target"], c.get("temperature", 1.0), c.get("entropy"))
    logp = torch.where(live, logp, 0.0)
    if h is not None:
        h = torch.where(live, h, 0.0)
    if c["op"] == "logprob":
        out = {"logp": logp, "lse": torch.where(live, lse, 0.0)}
        if c["entropy"]:
            out["entropy"] = h
        if c["backward"]:
            out["dlogits"] = _dlogits(s, p, lp, h, s["dlogp"], s["dentropy"] if c["entropy"] else None)
        return out
    if c["op"] == "policy":
        adv = s["advantage"]
        if c["sequences"]:
            adv = adv[torch.searchsorted(s["offsets"][1:], torch.arange(c["rows"], device="cuda", dtype=torch.int32), right=True)]
        w = live.float() / live.sum().clamp(min=1)
        r = torch.exp(logp - s["old_logp"])
        u, v = r * adv, torch.clamp(r, 1 - CLIP, 1 + CLIP) * adv
        loss = -torch.minimum(u, v)
        g = torch.where(u <= v, -u, 0.0)
        if c["kl"]:
            d = s["ref_logp"] - logp
            loss = loss + KL * (torch.exp(d) - d - 1)
            g = g + KL * (1 - torch.exp(d))
        gh = None
        if c["entropy"]:
            loss = loss - ENT * h
            gh = -ENT * w
        out = {"loss": (w * loss).sum(), "logp": logp, "dlogits": _dlogits(s, p, lp, h, w * g, gh)}
        if c["entropy"]:
            out["entropy"] = h
        return out
    seq = torch.searchsorted(s["offsets"][1:], torch.arange(c["rows"], device="cuda", dtype=torch.int32), right=True)
    per = 2 * c["pairs"]
    inside = seq[:, None] == torch.arange(per, device="cuda")
    sums = torch.where(inside, logp[:, None], 0.0).sum(0)
    share = torch.ones(per, device="cuda")
    if c["average"]:
        share = 1 / (inside & live[:, None]).sum(0).clamp(min=1).float()
        sums = sums * share
    # a long sequence's sum and its reference nearly cancel: the reference is taken off token by token, before the sum
    n = (inside & live[:, None]).sum(0).clamp(min=1).float()
    k = torch.where(inside & live[:, None], logp[:, None] - s["ref"] / (n * share), 0.0).sum(0) * share
    k = torch.where((inside & live[:, None]).any(0), k, -s["ref"])
    k = k[0::2] - k[1::2]
    if c["kind"] == "sigmoid":
        y = -BETA * k
        pair = torch.clamp(y, min=0) + torch.log1p(torch.exp(-y.abs()))
        g = -BETA / (1 + torch.exp(-y))
    elif c["kind"] == "hinge":
        pair = torch.clamp(1 - BETA * k, min=0)
        g = torch.where(BETA * k < 1, -BETA, 0.0)
    else:
        pair = (k - 0.5 / BETA) ** 2
        g = 2 * (k - 0.5 / BETA)
    g = (torch.stack([g, -g], 1).reshape(-1) / c["pairs"] * share)[seq]
    return {"loss": pair.sum() / c["pairs"], "pair_loss": pair, "logp": sums, "dlogits": _dlogits(s, p, None, None, g, None)}


# ------------------------------------------------------------------ in 64 bits

def _each(s, tau, f):
    """f(rows' slice, their log-probabilities in 64 bits), a slab of rows at a time."""
    rows, vocab = s["logits"].shape
    step = max(1, (1 << 27) // vocab)
    for a in range(0, rows, step):
        at = slice(a, min(rows, a + step))
        f(at, torch.log_softmax(s["logits"][at].double() / tau, 1))


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "clip":
        x = s["x"]
        norm = math.sqrt(math.fsum(float((a.double() * b.double()).sum()) for a, b in zip(x, s.get("y", x))))
        scale = min(1.0, s["max_norm"] / norm)
        if case["step"]:
            out = torch.cat([(w.double() - s["eta"] * scale * a.double()).reshape(-1) for w, a in zip(s["w"], x)])
        else:
            out = torch.cat([(scale * a.double()).reshape(-1) for a in x])
        return {"norm": torch.tensor([norm], dtype=torch.float64), "scale": torch.tensor([scale], dtype=torch.float64), "out": out}
    rows, tau = case["rows"], case.get("temperature", 1.0)
    live, target = s["target"] >= 0, s["target"].clamp(min=0)
    zero = lambda: torch.zeros(rows, dtype=torch.float64, device="cuda")  # noqa: E731
    logp, lse, h = zero(), zero(), zero()

    def stats(at, lp):
        logp[at] = lp.gather(1, target[at][:, None])[:, 0]
        lse[at] = torch.logsumexp(s["logits"][at].double() / tau, 1)
        if case.get("entropy"):
            h[at] = -torch.xlogy(lp.exp(), lp.exp()).sum(1)

    _each(s, tau, stats)
    logp[~live], lse[~live], h[~live] = 0, 0, 0
    g, gh = zero(), None
    if case["op"] == "logprob":
        out = {"logp": logp, "lse": lse}
        if case["entropy"]:
            out["entropy"] = h
        if not case["backward"]:
            return out
        g = s["dlogp"].double()
        gh = s["dentropy"].double() if case["entropy"] else None
    elif case["op"] == "policy":
        a = s["advantage"].double()
        if case["sequences"]:
            a = a.repeat_interleave(s["offsets"].long().diff())
        q = logp.clone().requires_grad_()
        ratio = torch.exp(q - s["old_logp"].double())
        inner = torch.where(a >= 0, torch.clamp(ratio, max=1 + CLIP), torch.clamp(ratio, min=1 - CLIP))
        loss = -a * inner
        if case["kl"]:
            d = s["ref_logp"].double() - q
            loss = loss + KL * (torch.expm1(d) - d)
        n = max(int(live.sum()), 1)
        loss = loss[live].sum() / n
        g = torch.autograd.grad(loss, q)[0]
        loss = loss.detach()
        out = {"loss": loss, "logp": logp}
        if case["entropy"]:
            out["loss"], out["entropy"] = loss - ENT * h.sum() / n, h
            gh = torch.full_like(h, -ENT / n)
    else:
        edges = s["offsets"].tolist()
        parts = [slice(a, b) for a, b in zip(edges, edges[1:])]
        count = [max(1, int(live[a].sum())) if case["average"] else 1 for a in parts]
        total = torch.stack([logp[a].sum() / n for a, n in zip(parts, count)])
        q = total.clone().requires_grad_()
        k = q - s["ref"].double()
        k = k[0::2] - k[1::2]
        pair = {"sigmoid": lambda: -torch.nn.functional.logsigmoid(BETA * k), "hinge": lambda: torch.relu(1 - BETA * k),
                "ipo": lambda: (k - 1 / (2 * BETA)).square()}[case["kind"]]()
        back = torch.autograd.grad(pair.mean(), q)[0]
        for a, n, v in zip(parts, count, back):
            g[a] = v / n
        out = {"loss": pair.mean().detach(), "pair_loss": pair.detach(), "logp": total}
    d = torch.empty(rows, case["vocab"], dtype=torch.float64, device="cuda")

    def back_rows(at, lp):
        p = lp.exp()
        y = p * -g[at][:, None]
        y.scatter_add_(1, target[at][:, None], g[at][:, None])
        if gh is not None:
            y -= gh[at][:, None] * (torch.xlogy(p, p) + p * h[at][:, None])
        y /= tau
        y[~live[at]] = 0
        d[at] = y

    _each(s, tau, back_rows)
    out["dlogits"] = d
    return out
