"""Operators behind the logits and the gradients of a model that is cut over the ranks.

What is measured, on one GPU that holds the p virtual ranks' buffers:

  logprobs           ra_token_logprobs: log probabilities of given tokens, the entropy and the
                     best alternatives, from logits whose vocabulary is split over the ranks
  logprobs_backward  ra_token_logprobs_backward: the gradient of the log probability and of
                     the entropy, from what the forward call left
  grad_norm          ra_grad_norm: the 2-norm over many gradient tensors
  grad_clip          ra_grad_clip: that norm, and every gradient scaled so that the norm of
                     all of them is at most max_norm
  allreduce_clip     ra_allreduce_clip: the ranks' gradients averaged or summed, clipped by
                     their norm, to every rank

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits (the
sums of squares in 64); with ``own`` true it calls the library.
"""

import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
CLIP_EPS = 1e-6              # added to the norm before max_norm is divided by it


# ---------------------------------------------------------------- cases

def listed():
    return [
        # serving, one sequence's next token: its log probability and five alternatives
        dict(name="logprobs 1x32000 p4 top5", op="logprobs", p=4, tokens=1, vocab=32000, valid=32000,
             dtype="float16", top=5, scale=1.0, masked=0.0),
        # serving, a batch's next tokens at a temperature of 0.8, a third of the columns masked
        dict(name="logprobs 16x128000 p8 top20", op="logprobs", p=8, tokens=16, vocab=128000, valid=128000,
             dtype="bfloat16", top=20, scale=1.25, masked=0.33),
        # the log probabilities of a long prompt's or of sampled answers' tokens, with alternatives
        dict(name="logprobs 4096x131072 p8 top20", op="logprobs", p=8, tokens=4096, vocab=131072, valid=131072,
             dtype="bfloat16", top=20, scale=1.0, masked=0.0),
        # a padded vocabulary that divides by nothing, 32-bit logits, many alternatives (distillation)
        dict(name="logprobs odd 1003x50017 p9 top64", op="logprobs", p=9, tokens=1003, vocab=50017, valid=50001,
             dtype="float32", top=64, scale=1.0, masked=0.0),
        # training on sampled answers: weights of log probability and entropy, back to the logits
        dict(name="logprobsbwd 4096x131072 p8", op="logprobs_backward", p=8, tokens=4096, vocab=131072,
             valid=131072, dtype="bfloat16", scale=1.0, entropy=True),
        # a small ragged batch of the same, without a bonus for entropy
        dict(name="logprobsbwd odd 517x50017 p9", op="logprobs_backward", p=9, tokens=517, vocab=50017,
             valid=50001, dtype="float32", scale=1.0, entropy=False),
        # a transformer's gradients, one tensor a parameter: the norm that is logged
        dict(name="norm 24 layers of 2048", op="grad_norm", layers=24, hidden=2048, vocab=32000,
             dtype="bfloat16", norms="float32", scale=1.0),
        # a small model, or an adapter: many small tensors, latency counts
        dict(name="norm 8 layers of 256", op="grad_norm", layers=8, hidden=256, vocab=1000,
             dtype="float32", norms="float32", scale=1.0),
        # clipping a transformer's gradients before the optimizer, of which it gets the clipped ones
        dict(name="clip 24 layers of 2048", op="grad_clip", layers=24, hidden=2048, vocab=32000,
             dtype="bfloat16", norms="float32", scale=1.0, wide=False),
        # odd sizes; 16-bit gradients of a scaled loss, unscaled and clipped into 32-bit ones
        dict(name="clip odd 6 layers of 517", op="grad_clip", layers=6, hidden=517, vocab=5003,
             dtype="float16", norms="float32", scale=1.0 / 1024, wide=True),
        # data parallel: a flat buffer of gradients on each of 8 ranks, averaged and clipped
        dict(name="allreduce clip 2^26 p8", op="allreduce_clip", p=8, n=1 << 26, dtype="float32",
             n_out=8, mean=True, scale=1.0),
        # a small odd buffer on 9 ranks, summed
        dict(name="allreduce clip 1000003 p9", op="allreduce_clip", p=9, n=1000003, dtype="bfloat16",
             n_out=9, mean=False, scale=1.0),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; odd as often as not."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:          # the multiples of 64 that most programs use
        n = n // 64 * 64 or n
    return max(lo, min(hi, n))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["logprobs", "logprobs", "logprobs_backward", "grad_norm", "grad_clip", "allreduce_clip"])
        dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        case = dict(op=op, dtype=dtype, scale=1.0)
        if op in ("logprobs", "logprobs_backward"):
            vocab = _log(rng, 1000, 160000)
            case |= dict(p=rng.choice([1, 2, 3, 4, 8, 8, 9, 16]), tokens=_log(rng, 1, 8192), vocab=vocab,
                         valid=vocab - rng.choice([0, 0, 17, 63]), scale=rng.choice([1.0, 1.0, 0.5, 1.25, 2.0]))
            if op == "logprobs":
                case |= dict(top=rng.choice([0, 1, 5, 20, 64]), masked=rng.choice([0.0, 0.0, 0.33]))
            else:
                case["entropy"] = rng.random() < 0.75
        elif op in ("grad_norm", "grad_clip"):
            case |= dict(layers=rng.randint(1, 32), hidden=_log(rng, 32, 2048), vocab=_log(rng, 100, 50000),
                         norms=rng.choice(["float32", dtype]), scale=rng.choice([1.0, 1.0, 0.25, 1.0 / 1024]))
            if op == "grad_clip":
                case["wide"] = rng.random() < 0.25
        else:
            p = rng.choice([1, 2, 3, 4, 8, 8, 9, 16])
            case |= dict(p=p, n=_log(rng, 1000, 1 << 28), n_out=rng.choice([1, p, p]), mean=rng.random() < 0.7,
                         scale=rng.choice([1.0, 1.0, 0.25]))
        # the plain forms hold several copies in 32 bits
        if work(case)["bytes"] <= most / 4:
            return case


# ---------------------------------------------------------------- inputs

def _bounds(n, p):
    """The library's partition: the first n mod p pieces hold one more."""
    return [i * (n // p) + min(i, n % p) for i in range(p + 1)]


def _zipf(vocab, n, g):
    """Token numbers as text gives them: the k-th about 1/k times as often as the first."""
    u = torch.rand(n, device="cuda", generator=g, dtype=torch.float64)
    return torch.exp(u * math.log(vocab + 1.0)).long().sub_(1).clamp_(0, vocab - 1)


def _shapes(case):
    """The parameters of a transformer: (shape, whether it is a norm's weight) for each."""
    h, v = case["hidden"], case["vocab"]
    kv, wide = max(1, h // 4), h * 8 // 3
    out = [((v, h), False)]
    for _ in range(case["layers"]):
        out += [((h,), True), ((h, h), False), ((kv, h), False), ((kv, h), False), ((h, h), False),
                ((h,), True), ((wide, h), False), ((wide, h), False), ((h, wide), False)]
    return out + [((h,), True), ((v, h), False)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = dict(case)

    def normal(*shape, dtype=dt, sigma=1.0):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        return x.normal_(0.0, sigma, generator=g)

    if op in ("logprobs", "logprobs_backward"):
        t, v, valid, p = case["tokens"], case["vocab"], case["valid"], case["p"]
        b = _bounds(v, p)
        s["ids"] = _zipf(valid, t, g)
        s["logits"] = []
        for r in range(p):
            x = normal(t, b[r + 1] - b[r], sigma=2.0)
            if case.get("masked"):
                x[torch.rand(x.shape, device="cuda", generator=g) < case["masked"]] = -math.inf
            at = s["ids"] - b[r]
            here = ((at >= 0) & (at < x.shape[1])).nonzero().squeeze(1)
            x[here, at[here]] = normal(len(here), sigma=1.0) + 8.0                 # a model that has learnt something
            s["logits"].append(x)
        f32 = dict(dtype=torch.float32, device="cuda")
        if op == "logprobs":
            s["ids"][torch.rand(t, device="cuda", generator=g) < 0.02] = -1            # tokens without one
            s["logprob"], s["entropy"], s["lse"] = (torch.empty(t, **f32) for _ in range(3))
            if case["top"]:
                s["top_ids"] = torch.empty((t, case["top"]), dtype=torch.int64, device="cuda")
                s["top_logprobs"] = torch.empty((t, case["top"]), **f32)
        else:
            # what the forward call leaves
            s["lse"], s["H"] = torch.empty(t, **f32), torch.empty(t, **f32)
            for lo in range(0, t, 256):
                y = torch.cat([x[lo:lo + 256] for x in s["logits"]], 1)[:, :valid].double() * case["scale"]
                lse = torch.logsumexp(y, 1)
                s["lse"][lo:lo + 256] = lse
                s["H"][lo:lo + 256] = lse - (torch.exp(y - lse[:, None]) * y).sum(1)
            s["dlogprob"] = normal(t, dtype=torch.float32, sigma=1.0)              # advantages
            s["dentropy"] = normal(t, dtype=torch.float32, sigma=0.01) if case["entropy"] else None
            s["grads"] = [torch.empty_like(x) for x in s["logits"]]
    elif op in ("grad_norm", "grad_clip"):
        s["tensors"] = []
        for i, (shape, is_norm) in enumerate(_shapes(case)):
            sigma = 1e-3 * 2.0 ** (i % 7 - 3) / case["scale"]                      # layers differ
            s["tensors"].append(normal(*shape, dtype=DTYPES[case["norms"]] if is_norm else dt, sigma=sigma))
        s["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
        s["max_norm"] = 1e-3 * math.sqrt(sum(x.numel() for x in s["tensors"])) / 2
        if op == "grad_clip":
            # a flat buffer for each type that an optimizer takes, one tensor's gradient behind the other's
            types = [torch.float32 if case["wide"] else x.dtype for x in s["tensors"]]
            s["flat"], s["outs"] = [], [None] * len(types)
            for dtype in dict.fromkeys(types):
                which = [i for i, t in enumerate(types) if t is dtype]
                sizes = [s["tensors"][i].numel() for i in which]
                s["flat"].append(torch.empty(sum(sizes), dtype=dtype, device="cuda"))
                for i, o in zip(which, s["flat"][-1].split(sizes)):
                    s["outs"][i] = o.view(s["tensors"][i].shape)
        if own:
            from ring_all_reduce_schedule_amd import binding as ra
            s["list"] = ra.TensorList(s["tensors"])
            s["out_list"] = ra.TensorList(s["outs"]) if op == "grad_clip" else None
    else:
        p, n = case["p"], case["n"]
        s["x"] = [normal(n, sigma=1e-3 / case["scale"]) for _ in range(p)]
        s["outs"] = [torch.empty_like(s["x"][0]) for _ in range(case["n_out"])]
        s["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
        s["max_norm"] = 1e-3 * math.sqrt(n / p if case["mean"] else n * p) / 2
        if own:
            from ring_all_reduce_schedule_amd import binding as ra
            s["ranks"] = ra.RankBuffers(s["x"])
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    from ring_all_reduce_schedule_amd import binding as ra
    op = s["op"]
    if op == "logprobs":
        ra.ra_token_logprobs(s["logits"], s["ids"], logprob=s["logprob"], entropy=s["entropy"], lse=s["lse"],
                             top_ids=s.get("top_ids"), top_logprobs=s.get("top_logprobs"), scale=s["scale"],
                             valid=s["valid"])
        return {"logprob": s["logprob"], "entropy": s["entropy"], "lse": s["lse"],
                "top_ids": s.get("top_ids"), "top_logprobs": s.get("top_logprobs")}
    if op == "logprobs_backward":
        ra.ra_token_logprobs_backward(s["logits"], s["ids"], s["lse"], s["grads"], dlogprob=s["dlogprob"],
                                      entropy=s["H"] if s["dentropy"] is not None else None,
                                      dentropy=s["dentropy"], scale=s["scale"], valid=s["valid"])
        return {"grads": s["grads"]}
    if op == "grad_norm":
        ra.ra_grad_norm(s["list"], s["norm"], scale=s["scale"])
        return {"norm": s["norm"]}
    if op == "grad_clip":
        ra.ra_grad_clip(s["list"], s["max_norm"], s["norm"], outs=s["out_list"], scale=s["scale"])
        return {"norm": s["norm"], "grads": s["flat"]}
    ra.ra_allreduce_clip(s["ranks"], s["max_norm"], s["norm"], s["outs"], op="avg" if s["mean"] else "sum",
                         scale=s["scale"])
    return {"norm": s["norm"], "grads": s["outs"]}


def _order(x):
    """Whole numbers that order like (x descending, column ascending)."""
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() << 32
    return key + torch.arange(x.shape[1] - 1, -1, -1, device=x.device)


def _coefficient(s, norm):
    return s["scale"] * (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)


def _plain(s):
    op = s["op"]
    if op in ("logprobs", "logprobs_backward"):
        x = torch.cat(s["logits"], 1)[:, :s["valid"]].float()
        at = s["ids"].clamp_min(0).unsqueeze(1)
        live = s["ids"] >= 0
    if op == "logprobs":
        y = x * s["scale"]
        y -= y.amax(1, keepdim=True)
        e = torch.exp(y)
        z = e.sum(1, keepdim=True)
        ln_z = torch.log(z)
        entropy = ln_z - torch.where(e > 0, e * y, 0.0).sum(1, keepdim=True) / z
        out = {"logprob": torch.where(live, (y.gather(1, at) - ln_z).squeeze(1), 0.0), "entropy": entropy.view(-1),
               "lse": (x.amax(1, keepdim=True) * s["scale"] + ln_z).view(-1), "top_ids": None, "top_logprobs": None}
        if s["top"]:
            best = torch.topk(_order(x), s["top"], dim=1).values & 0xffffffff
            out["top_ids"] = s["valid"] - 1 - best
            out["top_logprobs"] = y.gather(1, out["top_ids"]) - ln_z
        return out
    if op == "logprobs_backward":
        ln_p = x.mul_(s["scale"]).sub_(s["lse"].unsqueeze(1))
        a = torch.where(live, s["dlogprob"], 0.0).unsqueeze(1)
        d = torch.exp(ln_p).neg_()
        if s["dentropy"] is None:
            d *= a
        else:
            d *= a + s["dentropy"].unsqueeze(1) * (ln_p + s["H"].unsqueeze(1))
        d.scatter_add_(1, at, a)
        d = torch.nn.functional.pad(d.mul_(s["scale"]).to(s["logits"][0].dtype), (0, s["vocab"] - s["valid"]))
        return {"grads": [c.contiguous() for c in d.split([c.shape[1] for c in s["logits"]], 1)]}
    if op == "allreduce_clip":
        g = s["x"][0].float()
        for x in s["x"][1:]:
            g = g + x
        if s["mean"]:
            g = g / s["p"]
        tensors = [g.to(s["x"][0].dtype)]        # what an all-reduce leaves is of the buffers' type
    else:
        tensors = s["tensors"]
    squares = [torch.sum(x.float() * x.float(), dtype=torch.float64) for x in tensors]
    norm = s["scale"] * torch.sqrt(torch.stack(squares).sum())
    out = {"norm": norm.float().view(1)}
    if op == "grad_norm":
        return out
    c = _coefficient(s, norm).float()
    if op == "grad_clip":
        out["grads"] = [torch.cat([(x.float() * c).to(f.dtype).view(-1) for x, o in zip(s["tensors"], s["outs"])
                                   if o.dtype is f.dtype]) for f in s["flat"]]
    else:
        g = (tensors[0].float() * c).to(s["x"][0].dtype)
        out["grads"] = [g.clone() for _ in s["outs"]]
    return out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("logprobs", "logprobs_backward"):
        t, v = case["tokens"], case["valid"]
        if op == "logprobs":
            return {"bytes": t * v * e + 20 * t + 12 * t * case["top"], "flops": 8 * t * v}
        return {"bytes": t * (v + case["vocab"]) * e + (24 if case["entropy"] else 16) * t,
                "flops": (9 if case["entropy"] else 6) * t * v}
    if op == "allreduce_clip":
        return {"bytes": case["n"] * e * (case["p"] + case["n_out"]) + 4, "flops": case["n"] * (case["p"] + 3)}
    b = f = 0
    for shape, is_norm in _shapes(case):
        n = math.prod(shape)
        es = SIZE[case["norms"]] if is_norm else e
        b += n * es
        f += 2 * n
        if op == "grad_clip":
            b += n * (4 if case["wide"] else es)
            f += n
    return {"bytes": b + 4, "flops": f}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64

    def empty(*shape, dtype=f64):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op in ("logprobs", "logprobs_backward"):
        t, valid, scale, top = case["tokens"], case["valid"], case["scale"], case.get("top", 0)
        b = _bounds(case["vocab"], case["p"])
        if op == "logprobs":
            out = {"logprob": torch.zeros(t, dtype=f64, device="cuda"), "entropy": empty(t), "lse": empty(t),
                   "top_ids": empty(t, top, dtype=torch.int64) if top else None,
                   "top_logprobs": empty(t, top) if top else None}
        else:
            out = {"grads": [torch.zeros(x.shape, dtype=f64, device="cuda") for x in s["logits"]]}
        for lo in range(0, t, 256):
            hi = min(t, lo + 256)
            x = torch.cat([c[lo:hi] for c in s["logits"]], 1)[:, :valid].to(f64)
            ln_p = torch.log_softmax(scale * x, 1)
            ids = s["ids"][lo:hi]
            k = (ids >= 0).nonzero().squeeze(1)
            if op == "logprobs":
                out["lse"][lo:hi] = torch.logsumexp(scale * x, 1)
                out["logprob"][lo + k] = ln_p[k, ids[k]]
                out["entropy"][lo:hi] = torch.special.entr(torch.softmax(scale * x, 1)).sum(1)
                if top:
                    value, at = torch.sort(x, dim=1, descending=True, stable=True)
                    out["top_ids"][lo:hi] = at[:, :top]
                    out["top_logprobs"][lo:hi] = ln_p.gather(1, at[:, :top])
                continue
            # the definition's own derivative, with the statistics that the call is given
            ln_p = scale * x - s["lse"][lo:hi, None].to(f64)
            q = torch.exp(ln_p)
            d = -q * s["dlogprob"][lo:hi, None].to(f64)
            d[k, ids[k]] += s["dlogprob"][lo + k].to(f64)
            if case["entropy"]:
                d -= s["dentropy"][lo:hi, None].to(f64) * q * (ln_p + s["H"][lo:hi, None].to(f64))
            d = torch.nn.functional.pad(scale * d, (0, case["vocab"] - valid))
            for r in range(case["p"]):
                out["grads"][r][lo:hi] = d[:, b[r]:b[r + 1]]
        return out
    if op == "allreduce_clip":
        g = torch.zeros(case["n"], dtype=f64, device="cuda")
        for x in s["x"]:
            g += x
        tensors = [g / case["p"] if case["mean"] else g]
    else:
        tensors = s["tensors"]
    total = sum(float(torch.linalg.vector_norm(x.to(f64)) ** 2) for x in tensors)
    norm = case["scale"] * math.sqrt(total)
    out = {"norm": torch.tensor([norm], dtype=f64, device="cuda")}
    if op != "grad_norm":
        c = case["scale"] * min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        if op == "grad_clip":
            out["grads"] = [torch.cat([x.to(f64).flatten() * c for x, o in zip(tensors, s["outs"])
                                       if o.dtype is f.dtype]) for f in s["flat"]]
        else:
            out["grads"] = [tensors[0] * c] * case["n_out"]
    return out
