"""Operators at the places where a tensor-parallel transformer reduces over its ranks.

What is measured, on one GPU that holds the p virtual ranks' buffers:

  norm            ra_allreduce_rmsnorm: the ranks' partial sums folded, added to the
                  residual stream and normalised by their root mean square; the result
                  goes to every rank, in the buffers' type or in 8 bits with scales
  norm_backward   ra_allreduce_rmsnorm_backward: the ranks' partial gradients folded,
                  taken back through the norm, with the weight's gradient
  cross_entropy   ra_cross_entropy: softmax cross entropy over logits whose vocabulary
                  is split over the ranks, with its gradient
  embedding       ra_embedding: rows of a table whose vocabulary is split over the ranks
  embedding_backward  ra_embedding_backward: the gradient of those rows, by sorted tokens

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits;
with ``own`` true it calls the library.
"""

import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2, "float8": 1}
F8_MAX = 448.0               # the largest value of 8-bit e4m3
AMAX_FLOOR = 2.0 ** -110     # groups whose largest magnitude is smaller are scaled as if it were this
EPS = 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # decoding: one token leaves a row-parallel layer split over 8 ranks; latency is all there is
        dict(name="norm decode 1x4096 p8", op="norm", p=8, n_out=8, tokens=1, hidden=4096,
             dtype="bfloat16", residual="same", out="same", group=0),
        # prefill of a long prompt, the next layer's products in 8 bits (one scale a token)
        dict(name="norm prefill 4096x8192 p8 f8", op="norm", p=8, n_out=8, tokens=4096, hidden=8192,
             dtype="bfloat16", residual="same", out="float8", group=0),
        # odd sizes: rows that start on no vector boundary, 32-bit residual stream, one shared output
        # in 8 bits with a scale for every 128 columns
        dict(name="norm odd 1003x5001 p9 f8g", op="norm", p=9, n_out=1, tokens=1003, hidden=5001,
             dtype="float16", residual="float32", out="float8", group=128),
        # training: one layer's backward over a batch of 4096 tokens
        dict(name="normbwd 4096x8192 p8", op="norm_backward", p=8, n_out=1, tokens=4096, hidden=8192,
             dtype="bfloat16", residual="same"),
        # a small ragged batch in 32 bits
        dict(name="normbwd odd 517x2047 p4", op="norm_backward", p=4, n_out=0, tokens=517, hidden=2047,
             dtype="float32", residual="float32"),
        # training: the loss of 8192 tokens over a large vocabulary and its gradient, in one call
        dict(name="xent train 8192x131072 p8", op="cross_entropy", p=8, tokens=8192, vocab=131072,
             valid=131072, dtype="bfloat16", grad=True),
        # a padded vocabulary that divides by nothing, 32-bit logits
        dict(name="xent odd 1003x50017 p9", op="cross_entropy", p=9, tokens=1003, vocab=50017,
             valid=50001, dtype="float32", grad=True),
        # scoring a few tokens: the loss alone
        dict(name="xent score 4x128000 p8", op="cross_entropy", p=8, tokens=4, vocab=128000,
             valid=128000, dtype="bfloat16", grad=False),
        # decoding: the rows of 16 sequences' last tokens
        dict(name="embed decode 16x4096 p8", op="embedding", p=8, n_out=8, tokens=16, hidden=4096,
             vocab=32000, dtype="bfloat16"),
        # training: a batch's rows, to every rank
        dict(name="embed train 16384x4096 p8", op="embedding", p=8, n_out=8, tokens=16384, hidden=4096,
             vocab=131072, dtype="bfloat16"),
        # the gradient of that table, in 32 bits
        dict(name="embedbwd 16384x4096 p8", op="embedding_backward", p=8, tokens=16384, hidden=4096,
             vocab=131072, dtype="bfloat16", table="float32"),
        # a small odd table in 16 bits
        dict(name="embedbwd odd 1003x1001 p9", op="embedding_backward", p=9, tokens=1003, hidden=1001,
             vocab=5003, dtype="float16", table="float16"),
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
        op = rng.choice(["norm", "norm", "norm_backward", "cross_entropy", "cross_entropy",
                         "embedding", "embedding_backward"])
        p = rng.choice([1, 2, 3, 4, 8, 8, 9, 16])
        dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        tokens = _log(rng, 1, 16384)
        case = dict(op=op, p=p, tokens=tokens, dtype=dtype)
        if op == "norm":
            case |= dict(hidden=_log(rng, 64, 16384), n_out=rng.choice([1, p]),
                         residual=rng.choice(["none", "same", "same", "float32"]),
                         out=rng.choice(["same", "float8"]), group=0)
            if case["out"] == "float8":
                case["group"] = rng.choice([0, 32, 128])
        elif op == "norm_backward":
            case |= dict(hidden=_log(rng, 64, 16384), n_out=rng.choice([0, 1]),
                         residual=rng.choice(["same", "float32"]))
        elif op == "cross_entropy":
            vocab = _log(rng, 1000, 160000)
            case |= dict(vocab=vocab, valid=vocab - rng.choice([0, 0, 17, 63]), grad=rng.random() < 0.75)
        else:
            case |= dict(hidden=_log(rng, 64, 8192), vocab=_log(rng, 1000, 160000))
            if op == "embedding":
                case["n_out"] = rng.choice([1, p])
            else:
                case["table"] = rng.choice(["float32", dtype])
        # the plain forms hold several copies in 32 bits
        if work(case)["bytes"] <= most / 4:
            return case


# ---------------------------------------------------------------- inputs

def _residual_type(case):
    return case["dtype"] if case["residual"] == "same" else case["residual"]


def _bounds(n, p):
    """The library's partition: the first n mod p pieces hold one more."""
    return [i * (n // p) + min(i, n % p) for i in range(p + 1)]


def _zipf(vocab, n, g):
    """Token numbers as text gives them: the k-th about 1/k times as often as the first."""
    u = torch.rand(n, device="cuda", generator=g, dtype=torch.float64)
    return torch.exp(u * math.log(vocab + 1.0)).long().sub_(1).clamp_(0, vocab - 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, p, t = case["op"], case["p"], case["tokens"]
    dt = DTYPES[case["dtype"]]
    s = dict(case)

    def normal(*shape, dtype=dt, sigma=1.0):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        return x.normal_(0.0, sigma, generator=g)

    if op in ("norm", "norm_backward"):
        h = case["hidden"]
        s["x"] = normal(p, t, h, sigma=p ** -0.5)
        s["bufs"] = list(s["x"].unbind(0))
        s["weight"] = normal(h, dtype=torch.float32, sigma=0.1).add_(1.0).to(dt)
        wide = torch.ones(h, device="cuda")
        wide[torch.randint(0, h, (max(1, h // 500),), device="cuda", generator=g)] = 20.0   # outlier columns
        if case["residual"] != "none":
            rt = DTYPES[_residual_type(case)]
            s["stream"] = (normal(t, h, dtype=torch.float32) * wide).to(rt)
            s["stream_out"] = torch.empty_like(s["stream"])
    if op == "norm":
        ot = dt if case["out"] == "same" else torch.float8_e4m3fn
        s["y"] = torch.empty((case["n_out"], t, h), dtype=ot, device="cuda")
        s["outs"] = list(s["y"].unbind(0))
        if case["out"] == "float8":
            n = -(-h // case["group"]) if case["group"] else 1
            s["scale"] = torch.empty((case["n_out"], t, n), dtype=torch.float32, device="cuda")
            s["scales"] = list(s["scale"].unbind(0))
        s["rstd"] = torch.empty(t, dtype=torch.float32, device="cuda")
    elif op == "norm_backward":
        # h and 1/rms as the forward call leaves them, and the gradient that comes along the residual
        s["h"] = s.pop("stream")
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
        s["dh_in"] = normal(t, h, dtype=s["h"].dtype)
        s["dh"] = s.pop("stream_out")
        s["dx"] = torch.empty((case["n_out"], t, h), dtype=dt, device="cuda")
        s["dxs"] = list(s["dx"].unbind(0))
        s["dweight"] = torch.empty(h, dtype=torch.float32, device="cuda")
    elif op == "cross_entropy":
        v, valid = case["vocab"], case["valid"]
        b = _bounds(v, p)
        s["targets"] = _zipf(valid, t, g)
        s["targets"][torch.rand(t, device="cuda", generator=g) < 0.02] = -100      # tokens without a loss
        s["logits"], s["grads"] = [], []
        for r in range(p):
            x = normal(t, b[r + 1] - b[r], sigma=2.0)
            at = s["targets"] - b[r]
            here = ((at >= 0) & (at < x.shape[1])).nonzero().squeeze(1)
            x[here, at[here]] += 6.0                                               # a model that has learnt something
            s["logits"].append(x)
            s["grads"].append(torch.empty_like(x) if case["grad"] else None)
        s["loss"] = torch.empty(t, dtype=torch.float32, device="cuda")
        s["lse"] = torch.empty(t, dtype=torch.float32, device="cuda")
        s["dloss"] = torch.rand(t, device="cuda", generator=g)                     # weights of the tokens
    else:
        v, h = case["vocab"], case["hidden"]
        b = _bounds(v, p)
        s["ids"] = _zipf(v, t, g)
        s["ids"][torch.rand(t, device="cuda", generator=g) < 0.01] = -1            # padding
        s["scale"] = math.sqrt(h)
        if op == "embedding":
            s["table"] = normal(v, h, sigma=0.02)
            s["tables"] = [s["table"][b[r]:b[r + 1]] for r in range(p)]
            s["out"] = torch.empty((case["n_out"], t, h), dtype=dt, device="cuda")
            s["outs"] = list(s["out"].unbind(0))
        else:
            s["dy"] = normal(t, h, sigma=0.05)
            s["dtable"] = torch.empty((v, h), dtype=DTYPES[case["table"]], device="cuda")
            s["dtables"] = [s["dtable"][b[r]:b[r + 1]] for r in range(p)]
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    from ring_all_reduce_schedule_amd import binding as ra
    op = s["op"]
    if op == "norm":
        ra.ra_allreduce_rmsnorm(s["bufs"], s["weight"], EPS, s["outs"], residual=s.get("stream"),
                                residual_out=s.get("stream_out"), scales=s.get("scales"),
                                group=s["group"], rstd=s["rstd"])
        return {"y": s["y"], "scale": s.get("scale"), "h": s.get("stream_out"), "rstd": s["rstd"]}
    if op == "norm_backward":
        ra.ra_allreduce_rmsnorm_backward(s["bufs"], s["h"], s["rstd"], s["weight"], s["dh"],
                                         dh_in=s["dh_in"], dxs=s["dxs"], dweight=s["dweight"])
        return {"dh": s["dh"], "dx": s["dx"], "dweight": s["dweight"]}
    if op == "cross_entropy":
        ra.ra_cross_entropy(s["logits"], s["targets"], s["loss"], s["lse"], valid=s["valid"],
                            grads=s["grads"] if s["grad"] else None,
                            dloss=s["dloss"] if s["grad"] else None, grad_scale=1.0 / s["tokens"])
        return {"loss": s["loss"], "lse": s["lse"], "grads": s["grads"]}
    if op == "embedding":
        ra.ra_embedding(s["tables"], s["ids"], s["outs"], scale=s["scale"])
        return {"y": s["out"]}
    ra.ra_embedding_backward(s["dy"], s["ids"], s["dtables"], scale=s["scale"])
    return {"dtable": s["dtable"]}


def _plain(s):
    op = s["op"]
    if op == "norm":
        h = s["x"].sum(0, dtype=torch.float32)
        if "stream" in s:
            h = h + s["stream"]
        rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        y = h * rstd * s["weight"]
        scale = None
        if s["out"] == "float8":
            t, n = y.shape
            group = s["group"] or n
            full = torch.nn.functional.pad(y, (0, -n % group)).view(t, -1, group)
            scale = full.abs().amax(2, keepdim=True).clamp_min(AMAX_FLOOR) / F8_MAX
            y = (full / scale).view(t, -1)[:, :n]
            scale = scale.view(1, t, -1).repeat(s["n_out"], 1, 1)
        return {"y": y.to(s["y"].dtype).unsqueeze(0).repeat(s["n_out"], 1, 1), "scale": scale,
                "h": h.to(s["stream"].dtype) if "stream" in s else None, "rstd": rstd.view(-1)}
    if op == "norm_backward":
        dy = s["x"].sum(0, dtype=torch.float32)
        rstd = s["rstd"].unsqueeze(1)
        xhat = s["h"].float() * rstd
        gy = dy * s["weight"]
        dh = s["dh_in"] + rstd * (gy - xhat * (gy * xhat).mean(1, keepdim=True))
        return {"dh": dh.to(s["h"].dtype), "dx": dh.to(s["x"].dtype).unsqueeze(0).repeat(s["n_out"], 1, 1),
                "dweight": (dy * xhat).sum(0)}
    if op == "cross_entropy":
        x = torch.cat(s["logits"], 1)[:, :s["valid"]].float()
        m = x.amax(1, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(1, keepdim=True)
        lse = m + torch.log(z)
        live = s["targets"] >= 0
        at = s["targets"].clamp_min(0).unsqueeze(1)
        loss = torch.where(live, (lse - x.gather(1, at)).squeeze(1), 0.0)
        grads = [None] * s["p"]
        if s["grad"]:
            weight = torch.where(live, s["dloss"] / s["tokens"], 0.0).unsqueeze(1)
            d = e.div_(z).scatter_add_(1, at, torch.full_like(z, -1.0)).mul_(weight)
            d = torch.nn.functional.pad(d.to(s["logits"][0].dtype), (0, s["vocab"] - s["valid"]))
            grads = [c.contiguous() for c in d.split([x.shape[1] for x in s["logits"]], 1)]
        return {"loss": loss, "lse": lse.view(-1), "grads": grads}
    live = (s["ids"] >= 0).unsqueeze(1)
    at = s["ids"].clamp_min(0)
    if op == "embedding":
        y = torch.where(live, s["table"][at].float() * s["scale"], 0.0).to(s["table"].dtype)
        return {"y": y.unsqueeze(0).repeat(s["n_out"], 1, 1)}
    d = torch.zeros(s["dtable"].shape, dtype=torch.float32, device="cuda")
    d.index_add_(0, at, torch.where(live, s["dy"].float(), 0.0))
    return {"dtable": d.mul_(s["scale"]).to(s["dtable"].dtype)}


# ---------------------------------------------------------------- what a pass cannot do without

def _touched(t, v):
    """About how many rows t tokens touch, when the k-th comes with a chance of 1 / (k ln v)."""
    step, rows = math.log(v) / 200, 0.0
    for i in range(200):
        k = math.exp((i + 0.5) * step)
        rows += (1 - math.exp(-t / (k * math.log(v + 1.0)))) * k * step
    return int(rows) + 1


def work(case):
    op, p, t = case["op"], case["p"], case["tokens"]
    e = SIZE[case["dtype"]]
    if op == "norm":
        h = case["hidden"]
        n = -(-h // case["group"]) if case["group"] else 1
        res = 0 if case["residual"] == "none" else 2 * SIZE[_residual_type(case)]
        eo = e if case["out"] == "same" else 1
        b = t * h * (p * e + res + case["n_out"] * eo) + h * e + 4 * t
        if case["out"] == "float8":
            b += 4 * t * n * case["n_out"]
        return {"bytes": b, "flops": t * h * (p + 7)}
    if op == "norm_backward":
        h = case["hidden"]
        return {"bytes": t * h * (p * e + 3 * SIZE[_residual_type(case)] + case["n_out"] * e) + h * (e + 4) + 4 * t,
                "flops": t * h * (p + 12)}
    if op == "cross_entropy":
        v = case["valid"]
        b = t * v * e + 16 * t
        if case["grad"]:
            b += t * case["vocab"] * e + 4 * t
        return {"bytes": b, "flops": t * v * (8 if case["grad"] else 4)}
    h, v = case["hidden"], case["vocab"]
    if op == "embedding":
        rows = _touched(t, v)
        return {"bytes": rows * h * e + case["n_out"] * t * h * e + 8 * t, "flops": t * h}
    return {"bytes": t * h * e + v * h * SIZE[case["table"]] + 8 * t, "flops": t * h}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, p, t = case["op"], case["p"], case["tokens"]
    f64 = torch.float64
    if op == "norm":
        total = torch.zeros((t, case["hidden"]), dtype=f64, device="cuda")
        for b in s["bufs"]:
            total += b.to(f64)
        if "stream" in s:
            total += s["stream"].to(f64)
        power = torch.linalg.vector_norm(total, dim=1) ** 2 / case["hidden"]
        r = 1.0 / torch.sqrt(power + EPS)
        y = total * r[:, None] * s["weight"].to(f64)[None]
        scale = None
        if case["out"] == "float8":
            g = case["group"] or case["hidden"]
            parts = y.split(g, 1)
            scale = torch.stack([c.abs().max(1).values for c in parts], 1).clamp(min=AMAX_FLOOR) / F8_MAX
            y = torch.cat([c / scale[:, i:i + 1] for i, c in enumerate(parts)], 1)
            scale = scale.expand(case["n_out"], *scale.shape)
        return {"y": y.expand(case["n_out"], *y.shape), "scale": scale,
                "h": total if "stream" in s else None, "rstd": r}
    if op == "norm_backward":
        # h / rms(h) differentiated: (I - x x^T / n) / rms, with rms as the forward pass gave it
        n = case["hidden"]
        g = torch.zeros((t, n), dtype=f64, device="cuda")
        for b in s["bufs"]:
            g += b.to(f64)
        x = s["h"].to(f64) * s["rstd"].to(f64)[:, None]
        gw = g * s["weight"].to(f64)[None]
        along = torch.linalg.vecdot(gw, x, dim=1) / n
        d = s["dh_in"].to(f64) + (gw - along[:, None] * x) * s["rstd"].to(f64)[:, None]
        return {"dh": d, "dx": d.expand(case["n_out"], t, n), "dweight": torch.linalg.vecdot(g, x, dim=0)}
    if op == "cross_entropy":
        b = _bounds(case["vocab"], p)
        loss, lse = torch.zeros(t, dtype=f64, device="cuda"), torch.zeros(t, dtype=f64, device="cuda")
        grads = [torch.empty(g.shape, dtype=f64, device="cuda") for g in s["grads"] if g is not None]
        for lo in range(0, t, 1024):
            hi = min(t, lo + 1024)
            x = torch.cat([c[lo:hi].to(f64) for c in s["logits"]], 1)
            x[:, case["valid"]:] = -math.inf
            lse[lo:hi] = torch.logsumexp(x, 1)
            y = s["targets"][lo:hi]
            k = (y >= 0).nonzero().squeeze(1)
            loss[lo + k] = lse[lo + k] - x[k, y[k]]
            if grads:
                q = torch.exp(x - lse[lo:hi, None])
                q[k, y[k]] -= 1.0
                q *= (s["dloss"][lo:hi].to(f64) / t * (y >= 0))[:, None]
                for r in range(p):
                    grads[r][lo:hi] = q[:, b[r]:b[r + 1]]
        return {"loss": loss, "lse": lse, "grads": grads or None}
    if op == "embedding":
        b = _bounds(case["vocab"], p)
        y = torch.zeros((t, case["hidden"]), dtype=f64, device="cuda")
        for r in range(p):
            k = ((s["ids"] >= b[r]) & (s["ids"] < b[r + 1])).nonzero().squeeze(1)
            y[k] = s["tables"][r][s["ids"][k] - b[r]].to(f64) * s["scale"]
        return {"y": y.expand(case["n_out"], *y.shape)}
    k = (s["ids"] >= 0).nonzero().squeeze(1)
    rows, to = torch.unique(s["ids"][k], return_inverse=True)
    sums = torch.zeros((rows.numel(), case["hidden"]), dtype=f64, device="cuda")
    sums.index_add_(0, to, s["dy"][k].to(f64))
    d = torch.zeros((case["vocab"], case["hidden"]), dtype=f64, device="cuda")
    d[rows] = sums * s["scale"]
    return {"dtable": d}
