"""What is measured of the 8-bit checkpoints and of the verification of drafts.

Each case is one pass: a matrix kept in 8 bits and restored (`checkpoint`), a
layer's weight gradient from the checkpoint of its input and the output gradient
that arrives (`weight_grad`), the running average of a factor from a checkpoint
(`factor`), and the verification of drafted tokens (`verify`).  Where `own` is
false, `run` computes it in elementary torch operations in 32 bits; where it is
true, it calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the single fully connected layer's input at 32 samples, with the column of ones of its bias (latency)
        {"name": "checkpoint small", "op": "checkpoint", "rows": 32, "cols": 64, "dtype": "f32", "one": True},
        # a ragged batch of tokens, an odd width: every row on another alignment
        {"name": "checkpoint odd", "op": "checkpoint", "rows": 5003, "cols": 2049, "dtype": "f16", "one": False},
        # the input of a wide layer over a long batch of tokens
        {"name": "checkpoint large", "op": "checkpoint", "rows": 32768, "cols": 8192, "dtype": "bf16", "one": False},
        # the single fully connected layer, 64 -> 32 with a bias (latency)
        {"name": "weight_grad small", "op": "weight_grad", "rows": 32, "cols": 64, "outs": 32, "dtype": "f32", "one": True},
        # a classifier's output layer, 2048 -> 1000 with a bias, over a ragged batch
        {"name": "weight_grad output layer", "op": "weight_grad", "rows": 1027, "cols": 2048, "outs": 1000, "dtype": "f16", "one": True},
        # a square layer over a long batch of tokens
        {"name": "weight_grad large", "op": "weight_grad", "rows": 16384, "cols": 4096, "outs": 8192, "dtype": "bf16", "one": False},
        # the factor of the small layer's input (latency)
        {"name": "factor small", "op": "factor", "rows": 32, "cols": 64, "one": True, "packed": False},
        # the factor of a wide layer's input with its bias, stored packed
        {"name": "factor large", "op": "factor", "rows": 8192, "cols": 4096, "one": True, "packed": True},
        # one request that decodes with four drafted tokens (latency)
        {"name": "verify one", "op": "verify", "seqs": 1, "drafts": 4, "ragged": False, "vocab": 131072, "dtype": "bf16", "draft": "rows",
         "greedy": False, "temperature": 1.0},
        # a few requests decoded greedily, drafts looked up in the text so far
        {"name": "verify greedy", "op": "verify", "seqs": 12, "drafts": 5, "ragged": True, "vocab": 32768, "dtype": "f16", "draft": "none",
         "greedy": True, "temperature": 1.0},
        # ragged drafts, some sequences without any, an odd vocabulary, the draft's sums kept from drafting
        {"name": "verify odd", "op": "verify", "seqs": 37, "drafts": 7, "ragged": True, "vocab": 50001, "dtype": "f32", "draft": "saved",
         "greedy": False, "temperature": 0.8},
        # a rollout's whole batch over a large vocabulary
        {"name": "verify batch", "op": "verify", "seqs": 256, "drafts": 7, "ragged": False, "vocab": 131072, "dtype": "bf16", "draft": "rows",
         "greedy": False, "temperature": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["checkpoint", "weight_grad", "factor", "verify", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "checkpoint":
        cols = _log(rng, 1, 20_000)
        return {"op": op, "rows": _log(rng, 1, min(100_000, 250_000_000 // (cols * SIZE[dtype]) * 2)), "cols": cols, "dtype": dtype,
                "one": rng.random() < 0.3}
    if op == "weight_grad":
        cols, outs = _log(rng, 8, 9000), _log(rng, 8, 9000)
        rows = _log(rng, 1, min(20_000, 500_000_000_000 // (cols * outs)))
        return {"op": op, "rows": rows, "cols": cols, "outs": outs, "dtype": dtype, "one": rng.random() < 0.4}
    if op == "factor":
        cols = _log(rng, 8, 8000)
        return {"op": op, "rows": _log(rng, 1, min(30_000, 300_000_000_000 // (cols * cols))), "cols": cols, "one": rng.random() < 0.4,
                "packed": rng.random() < 0.5}
    vocab = _log(rng, 16, 200_000)
    drafts = rng.randint(0, 12)
    seqs = _log(rng, 1, max(1, min(500, 250_000_000 // (vocab * (drafts + 1)) * 2 // SIZE[dtype])))
    greedy = rng.random() < 0.25
    return {"op": op, "seqs": seqs, "drafts": drafts, "ragged": rng.random() < 0.6, "vocab": vocab, "dtype": dtype,
            "draft": rng.choice(["rows", "rows", "saved", "none"]) if not greedy else "none", "greedy": greedy,
            "temperature": rng.choice([1.0, 1.0, 0.7, 1.3])}


def work(case):
    """Bytes that each input is read and each output written once (a verification:
    of the rows up to the first token that is not accepted, at 7 of 10 accepted),
    and the operations."""
    if case["op"] == "verify":
        k, v, e = case["drafts"] / 2 if case["ragged"] else case["drafts"], case["vocab"], SIZE[case["dtype"]]
        rows = case["seqs"] * (1 - 0.7 ** (k + 1)) / 0.3
        read = rows * v * e  # the target's
        if case["draft"] == "rows":
            read += min(rows, case["seqs"] * k) * v * e
        elif case["draft"] == "saved":
            read += case["seqs"] * (1 - 0.7 ** k) * v * e
        if not case["greedy"]:
            read += case["seqs"] * v * 4
        return {"bytes": read + case["seqs"] * (k + 1) * 20, "flops": rows * v * 4}
    rows, width = case["rows"], case["cols"] + case["one"]
    if case["op"] == "checkpoint":  # kept in 8 bits and a byte for each 32, read back
        n = rows * case["cols"]
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 2 * rows * width * 33 / 32, "flops": 4 * n}
    if case["op"] == "weight_grad":
        n = rows * case["outs"]
        return {"bytes": rows * width * 33 / 32 + n * SIZE[case["dtype"]] + 2 * n * 33 / 32 + 4 * case["outs"] * width,
                "flops": 2 * n * width}
    return {"bytes": rows * width * 33 / 32 + 4 * width * (width + 1), "flops": rows * width * (width + 1)}


# ------------------------------------------------------------------ 8 bits

def _block_exponent(amax):
    """The smallest e with amax <= 448 2^e, at least -127."""
    mant, exp = torch.frexp(amax)  # amax = mant 2^exp, 0.5 <= mant < 1
    e = exp - 9 + (mant > 0.875)
    return torch.where(amax > 0, e, -127).clamp(min=-127)


def _quantise(x, one):
    """Elements (e4m3) and exponents of blocks of 32 rows of each column of x, in 32
    bits, with a last column of ones where `one`."""
    x = x.float()
    if one:
        x = torch.cat([x, torch.ones_like(x[:, :1])], 1)
    rows, cols = x.shape
    x = torch.cat([x, x.new_zeros(-rows % 32, cols)]).view(-1, 32, cols)
    e = _block_exponent(x.abs().amax(1))
    q = torch.ldexp(x, -e[:, None]).to(torch.float8_e4m3fn)
    return q.view(-1, cols)[:rows], e


def _values(q, e):
    """What elements and exponents stand for, in 32 bits."""
    rows = q.shape[0]
    return torch.ldexp(q.float(), e.repeat_interleave(32, 0)[:rows])


def _tiles(e, rows):
    """Exponents in the order that the library keeps them in: 512 bytes for 128 columns
    and 128 rows, a column's four blocks next to one another, columns 32 apart next to
    those."""
    blocks, cols = e.shape
    chunks, wide = -(-rows // 128), -(-cols // 128)
    b = torch.zeros(4 * chunks, 128 * wide, dtype=torch.uint8, device=e.device)
    b[:blocks, :cols] = (e + 127).to(torch.uint8)
    return b.view(chunks, 4, wide, 4, 32).permute(2, 0, 4, 3, 1).contiguous().view(-1)


def _untiled(b, rows, cols):
    """The exponents of _tiles."""
    chunks, wide = -(-rows // 128), -(-cols // 128)
    e = b.view(wide, chunks, 32, 4, 4).permute(1, 4, 0, 3, 2).reshape(4 * chunks, 128 * wide)
    return e[:-(-rows // 32), :cols].to(torch.int32) - 127


def _buffers(rows, cols):
    """Room for a checkpoint: elements on a pitch of 16 bytes, and the exponents."""
    return (torch.empty(rows, -(-cols // 16) * 16, dtype=torch.uint8, device="cuda"),
            torch.empty(-(-rows // 128) * -(-cols // 128) * 512, dtype=torch.uint8, device="cuda"))


def _checkpoint(x, one):
    """A checkpoint that a forward pass has left behind."""
    q, e = _quantise(x, one)
    elems, scales = _buffers(*q.shape)
    elems[:, :q.shape[1]] = q.view(torch.uint8)
    scales.copy_(_tiles(e, q.shape[0]))
    return elems, scales


# ------------------------------------------------------------------ the inputs

def _activations(rows, cols, gen, dtype):
    """A layer's input: rectified, with some channels far above the others."""
    channel = torch.exp(1.5 * torch.randn(cols, device="cuda", generator=gen))
    x = torch.empty(rows, cols, dtype=dtype, device="cuda")
    step = max(32, (1 << 27) // cols)
    for a in range(0, rows, step):
        n = min(rows, a + step) - a
        x[a:a + n] = torch.relu(torch.randn(n, cols, device="cuda", generator=gen) + 0.3) * channel
    return x


def _gradients(rows, cols, gen, dtype):
    """Output gradients: tokens whose gradients differ by orders of magnitude."""
    token = torch.exp(2.0 * torch.randn(rows, 1, device="cuda", generator=gen)) * 1e-3
    return (torch.randn(rows, cols, device="cuda", generator=gen) * token).to(dtype)


def _drafts(case, gen, s):
    """The target's logits as a language model's are, a draft model's near them, and the
    tokens that the draft model chose."""
    vocab, dt, tau = case["vocab"], DTYPES[case["dtype"]], case["temperature"]
    most = case["drafts"] + 1
    n = torch.full((case["seqs"],), most, device="cuda")
    if case["ragged"]:
        n = 1 + (torch.arange(case["seqs"], device="cuda") * 7 + 3) % most  # every number of drafts, none among them
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), n.cumsum(0)])
    s["offsets"] = off.to(torch.int32)
    rows = int(off[-1])
    bias = -2.0 * torch.log(torch.arange(1, vocab + 1, device="cuda", dtype=torch.float32))
    bias = (bias - bias.mean())[torch.randperm(vocab, device="cuda", generator=gen)]
    s["logits"] = torch.empty(rows, vocab, dtype=dt, device="cuda")
    drafted = torch.empty_like(s["logits"]) if case["draft"] != "none" else None
    s["tokens"] = torch.empty(rows, dtype=torch.int64, device="cuda")
    saved = torch.empty(rows, 2, device="cuda")
    step = max(1, (1 << 27) // vocab)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        x = torch.randn(b - a, vocab, device="cuda", generator=gen).mul_(1.5).add_(bias)
        s["logits"][a:b] = x
        x = (x + 0.5 * torch.randn(x.shape, device="cuda", generator=gen)).to(dt)
        if drafted is not None:
            drafted[a:b] = x
        x = x.float()
        saved[a:b, 0] = x.amax(1)
        saved[a:b, 1] = torch.exp(((x - x.amax(1, keepdim=True)) / tau).double()).sum(1).float()
        if not case["greedy"]:  # drawn from the draft's distribution
            x = x / tau - torch.empty_like(x).exponential_(generator=gen).log_()
        s["tokens"][a:b] = x.argmax(1)
        del x
    if drafted is not None:
        s["draft"] = drafted
    if case["draft"] == "saved":
        s["saved"] = saved
    if not case["greedy"]:
        s["uniform"] = torch.rand(rows, device="cuda", generator=gen)
        s["noise"] = torch.empty(case["seqs"], vocab, device="cuda").exponential_(generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "verify":
        _drafts(case, gen, s)
        return s
    rows, cols, one = case["rows"], case["cols"], case["one"]
    if case["op"] == "checkpoint":
        s["x"] = _activations(rows, cols, gen, DTYPES[case["dtype"]])
        s["q"], s["scales"] = _buffers(rows, cols + one)
        s["out"] = torch.empty_like(s["x"])
        return s
    s["q"], s["scales"] = _checkpoint(_activations(rows, cols, gen, torch.bfloat16), one)
    if case["op"] == "weight_grad":
        s["g"] = _gradients(rows, case["outs"], gen, DTYPES[case["dtype"]])
        s["gq"], s["gscales"] = _buffers(rows, case["outs"])
        s["dw"] = torch.empty(case["outs"], cols + one, device="cuda")
        return s
    d = cols + one
    s["F"] = torch.eye(d, device="cuda")  # where the running average starts
    if case["packed"]:
        i = torch.triu_indices(d, d, device="cuda")
        s["F"] = s["F"][i[0], i[1]].contiguous()
    return s


# ------------------------------------------------------------------ the passes

XI = 0.95


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from second_order_optimisation_gb300 import kfac
    c = s["case"]
    if c["op"] == "verify":
        rows = len(s["tokens"])
        accepted = torch.empty(c["seqs"], dtype=torch.int32, device="cuda")
        tokens, logp = torch.empty_like(s["tokens"]), torch.empty(rows, device="cuda")
        kfac.kfac_verify_draft(kfac.VerifyDraft(
            s["logits"], s["tokens"], s["offsets"], accepted, tokens, logp, draft=s.get("draft"), draft_saved=s.get("saved"),
            uniform=s.get("uniform"), noise=s.get("noise"), greedy=c["greedy"], temperature=c["temperature"],
            draft_temperature=c["temperature"]))
        return {"accepted": accepted, "tokens": tokens, "logp": logp}
    rows, width = c["rows"], c["cols"] + c["one"]
    a = kfac.Checkpoint(s["q"], s["scales"], rows, width)
    if c["op"] == "checkpoint":
        kfac.kfac_checkpoint_store([kfac.CheckpointItem(s["x"], a, append_one=c["one"])])
        kfac.kfac_checkpoint_load([kfac.CheckpointItem(s["out"], a, append_one=c["one"])])
        return {"x": s["out"]}
    if c["op"] == "weight_grad":
        g = kfac.Checkpoint(s["gq"], s["gscales"], rows, c["outs"])
        kfac.kfac_checkpoint_store([kfac.CheckpointItem(s["g"], g)])
        kfac.kfac_weight_grad([kfac.WeightGrad(a, g, s["dw"], alpha=1.0 / rows)])
        return {"dw": s["dw"]}
    kfac.kfac_factor_update([kfac.FactorSource(a, s["F"], alpha=(1 - XI) / rows, beta=XI, packed=c["packed"])])
    return {"F": s["F"]}


def _log_probs(z, tau):
    x = z / tau if tau != 1.0 else z
    x = x - x.amax(1, keepdim=True)
    return x - torch.log(torch.exp(x).sum(1, keepdim=True))


def _first(mask):
    """The lowest index of a true value in each row."""
    n = mask.shape[1]
    return torch.where(mask, torch.arange(n, device=mask.device), n).amin(1)


def _plain_verify(s):
    c, off, tok = s["case"], s["offsets"].long(), s["tokens"]
    rows, seqs, tau = len(tok), c["seqs"], c["temperature"]
    at = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(off[1:], at, right=True)
    lp = _log_probs(s["logits"].float(), tau)
    if c["greedy"]:
        best = _first(s["logits"] == s["logits"].amax(1, keepdim=True))
        ok = tok == best
    else:
        # next to a border 32 bits are too few
        lpt = _log_probs_of(s["logits"], tok, tau)
        ratio = torch.exp(lpt if "draft" not in s else lpt - _log_probs_of(s["draft"], tok, tau))
        ok = s["uniform"].double() < ratio
    bonus = at == off[1:][seq] - 1
    stop = torch.where(ok & ~bonus, rows, at)
    row = torch.full((seqs,), rows, device="cuda").scatter_reduce(0, seq, stop, "amin")
    accepted = row - off[:-1]
    if c["greedy"]:
        new = best[row]
    else:
        p = torch.exp(_log_probs(s["logits"][row].double(), tau))
        if "draft" in s:
            q = torch.exp(_log_probs(s["draft"][row].double(), tau))
        else:
            q = torch.zeros_like(p).scatter_(1, tok[row][:, None], 1.0)
        p = torch.where(bonus[row][:, None], p, torch.clamp(p - q, min=0))
        key = p / s["noise"]
        new = _first(key == key.amax(1, keepdim=True))
    out = torch.where(at < row[seq], tok, -1)
    out[row] = new
    logp = torch.where(out >= 0, lp.gather(1, out.clamp(min=0)[:, None])[:, 0], 0.0)
    return {"accepted": accepted.to(torch.int32), "tokens": out, "logp": logp}


def _log_probs_of(z, tok, tau):
    """The log-probability of each row's token in 64 bits."""
    x = z.float()
    m = x.amax(1, keepdim=True)
    total = torch.exp((x - m) / tau).sum(1, dtype=torch.float64)
    return ((x.gather(1, tok[:, None]) - m)[:, 0]).double() / tau - torch.log(total)


def _plain(s):
    c = s["case"]
    if c["op"] == "verify":
        return _plain_verify(s)
    if c["op"] == "checkpoint":
        x = _values(*_quantise(s["x"], c["one"]))
        s["out"].copy_(x[:, :c["cols"]])
        return {"x": s["out"]}
    rows, width = c["rows"], c["cols"] + c["one"]
    a = _values(s["q"][:, :width].view(torch.float8_e4m3fn), _untiled(s["scales"], rows, width))
    if c["op"] == "weight_grad":
        g = _values(*_quantise(s["g"], False))
        s["dw"].copy_(g.t() @ a / rows)
        return {"dw": s["dw"]}
    f = a.t() @ a * ((1 - XI) / rows)
    i = torch.triu_indices(width, width, device="cuda")
    f = f[i[0], i[1]]
    if c["packed"]:
        s["F"].mul_(XI).add_(f)
    else:
        s["F"][i[0], i[1]] = XI * s["F"][i[0], i[1]] + f
    return {"F": s["F"]}


# ------------------------------------------------------------------ in 64 bits

def _rounded(x):
    """x [rows, cols] as its 8-bit form stands for it: e4m3 has steps of 2^-3 of a value's
    binade, at least 2^-9, and blocks of 32 rows share a power of two."""
    x = x.double()
    rows, cols = x.shape
    out = torch.empty_like(x)
    for a in range(0, rows, 32):
        b = x[a:a + 32]
        top = b.abs().amax(0)
        e = torch.ceil(torch.log2(top / 448))
        e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)  # where the logarithm was rounded up
        e = torch.where(top > 448 * torch.exp2(e), e + 1, e).clamp(min=-127)
        e = torch.where(top > 0, e, -127.0)
        y = b / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        out[a:a + 32] = torch.round(y / step) * step * torch.exp2(e)
    return out


def _kept(q, scales, rows, width):
    """The values of a kept checkpoint, bit by bit."""
    b = q[:, :width].to(torch.int64)
    sign, exp, man = 1.0 - 2.0 * (b >> 7).double(), (b >> 3) & 15, (b & 7).double()
    v = torch.where(exp > 0, (8 + man) * torch.exp2((exp - 10).double()), man * 2.0 ** -9) * sign
    r, c = torch.arange(rows, device="cuda")[:, None], torch.arange(width, device="cuda")[None]
    at = ((c // 128) * -(-rows // 128) + r // 128) * 512 + (c % 32) * 16 + c % 128 // 32 * 4 + r % 128 // 32
    return v * torch.exp2(scales[at].double() - 127)


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, s)
    if case["op"] == "checkpoint":
        return {"x": _rounded(s["x"])}
    rows, width = case["rows"], case["cols"] + case["one"]
    a = _kept(s["q"], s["scales"], rows, width)
    if case["op"] == "weight_grad":
        return {"dw": torch.einsum("mo,mi->oi", _rounded(s["g"]), a) / rows}
    f = torch.einsum("mi,mj->ij", a, a) * ((1 - XI) / rows)
    if case["packed"]:
        f += XI * torch.eye(width, dtype=torch.float64, device="cuda")
        return {"F": torch.cat([f[i, i:] for i in range(width)])}
    f = torch.triu(f) + XI * torch.eye(width, dtype=torch.float64, device="cuda")
    return {"F": f}


def _exact_verify(case, s):
    off, tok, tau = s["offsets"].tolist(), s["tokens"].tolist(), case["temperature"]
    accepted, tokens, logp = [], [-1] * len(tok), torch.zeros(len(tok), dtype=torch.float64, device="cuda")
    for b, (lo, hi) in enumerate(zip(off, off[1:])):
        lp = torch.log_softmax(s["logits"][lo:hi].double() / tau, 1)
        lq = torch.log_softmax(s["draft"][lo:hi].double() / tau, 1) if "draft" in s else None
        n = 0
        while n < hi - lo - 1:
            x = tok[lo + n]
            if case["greedy"]:
                if int((lp[n] == lp[n].max()).nonzero()[0]) != x:
                    break
            elif not float(s["uniform"][lo + n]) * (float(lq[n, x].exp()) if lq is not None else 1.0) < float(lp[n, x].exp()):
                break
            tokens[lo + n] = x
            logp[lo + n] = lp[n, x]
            n += 1
        if case["greedy"]:
            new = int((lp[n] == lp[n].max()).nonzero()[0])
        else:
            r = lp[n].exp()
            if n < hi - lo - 1:
                if lq is not None:
                    r = torch.relu(r - lq[n].exp())
                else:
                    r[tok[lo + n]] = 0
            new = int((torch.log(r) - torch.log(s["noise"][b].double())).argmax())
        tokens[lo + n] = new
        logp[lo + n] = lp[n, new]
        accepted.append(n)
    return {"accepted": torch.tensor(accepted, dtype=torch.int32), "tokens": torch.tensor(tokens), "logp": logp}
