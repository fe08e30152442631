"""The operators of a parallel fine-tuning step whose result involves the other ranks, as cases to measure:
dropout after a row-parallel layer's AllReduce (bias, a mask drawn by counter and never stored, residual) and its
gradients; the tokens' log-probabilities from logits whose vocabulary is cut over the ranks, and their gradient;
the clipped policy loss with a KL term over every rank's tokens, with its gradient.

Where `own` is false `run` computes them from elementary torch operations; where it is true it calls
the library.  Layouts are the same either way."""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
SIZE = {"float32": 4, "float16": 2, "bfloat16": 2}
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.05


def listed():
    return [
        # a small model's hidden states on 4 ranks: latency
        {"name": "dropout_small", "op": "dropout", "ranks": 4, "rows": 64, "ragged": False, "cols": 768,
         "dtype": "float32", "wtype": "float32", "pad": 0, "p": 0.1, "residual": True, "replicas": True},
        # ragged batches on 8 data-parallel ranks, an odd width inside padded rows, bias in 32 bits
        {"name": "dropout_ragged", "op": "dropout", "ranks": 8, "rows": 1500, "ragged": True, "cols": 4097,
         "dtype": "float16", "wtype": "float32", "pad": 9, "p": 0.2, "residual": True, "replicas": False},
        # a training step's whole batch on 8 ranks
        {"name": "dropout_batch", "op": "dropout", "ranks": 8, "rows": 4096, "ragged": False, "cols": 8192,
         "dtype": "bfloat16", "wtype": "bfloat16", "pad": 0, "p": 0.1, "residual": True, "replicas": False},
        # the backward pass of ragged batches and an odd width, the bias gradient in 32 bits
        {"name": "dropout_backward_ragged", "op": "dropout_backward", "ranks": 8, "rows": 700, "ragged": True,
         "cols": 2047, "dtype": "float16", "wtype": "float32", "pad": 0, "p": 0.1, "replicas": False},
        # a training step's whole batch on 8 ranks
        {"name": "dropout_backward_batch", "op": "dropout_backward", "ranks": 8, "rows": 4096, "ragged": False,
         "cols": 8192, "dtype": "bfloat16", "wtype": "bfloat16", "pad": 0, "p": 0.1, "replicas": False},
        # one generated token scored while serving, a vocabulary of 128000 over 8 ranks: latency
        {"name": "logprob_token", "op": "logprob", "ranks": 8, "rows": 1, "cols": 16000, "uneven": False,
         "dtype": "bfloat16", "scale": 1.0, "ignored": 0.0},
        # a sequence whose prompt is not scored, uneven odd shards, logits in 32 bits, a sampling temperature
        {"name": "logprob_ragged", "op": "logprob", "ranks": 5, "rows": 700, "cols": 10007, "uneven": True,
         "dtype": "float32", "scale": 1.25, "ignored": 0.3},
        # a training step's tokens, a vocabulary of 128000 over 8 ranks
        {"name": "logprob_batch", "op": "logprob", "ranks": 8, "rows": 8192, "cols": 16000, "uneven": False,
         "dtype": "bfloat16", "scale": 1.0, "ignored": 0.0},
        # a short sequence's gradient, uneven odd shards, the prompt's rows zero
        {"name": "logprob_backward_small", "op": "logprob_backward", "ranks": 4, "rows": 96, "cols": 8003,
         "uneven": True, "dtype": "float32", "scale": 1.25, "ignored": 0.3},
        # a training step's tokens
        {"name": "logprob_backward_batch", "op": "logprob_backward", "ranks": 8, "rows": 8192, "cols": 16000,
         "uneven": False, "dtype": "bfloat16", "scale": 1.0, "ignored": 0.0},
        # a few short sequences on 4 ranks: latency
        {"name": "policy_small", "op": "policy", "ranks": 4, "tokens": 500, "ragged": True, "kl": True},
        # every token of a large batch on 8 ranks
        {"name": "policy_batch", "op": "policy", "ranks": 8, "tokens": 262144, "ragged": False, "kl": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["dropout", "dropout_backward", "logprob", "logprob_backward", "policy"])
    ranks = rng.choice([1, 1, 2, 3, 4, 8, 8, 16, 20])
    if op == "policy":
        return {"op": op, "ranks": ranks, "tokens": _log(rng, 1, 2097152 // ranks), "ragged": rng.random() < 0.6,
                "kl": rng.random() < 0.7}
    dtype = rng.choice(["float32", "float16", "bfloat16"])
    most = 1 << (26 if dtype == "float32" else 27)
    if op in ("dropout", "dropout_backward"):
        cols = _log(rng, 8, 40000)
        if rng.random() < 0.5:
            cols = max(8, cols // 64 * 64)
        case = {"op": op, "ranks": ranks, "rows": _log(rng, 1, max(1, min(20000, most // (cols * ranks)))),
                "ragged": rng.random() < 0.5, "cols": cols, "dtype": dtype, "wtype": rng.choice([dtype, "float32"]),
                "pad": rng.choice([0, 0, 8, 3]), "p": rng.choice([0.05, 0.1, 0.2, 0.5])}
        if op == "dropout":
            case["residual"] = rng.random() < 0.8
        case["replicas"] = not case["ragged"] and rng.random() < 0.4
        return case
    cols = _log(rng, 32, 160000 // ranks)
    if rng.random() < 0.5:
        cols = max(32, cols // 64 * 64)
    return {"op": op, "ranks": ranks, "rows": _log(rng, 1, max(1, min(20000, most // (cols * ranks)))), "cols": cols,
            "uneven": rng.random() < 0.5, "dtype": dtype, "scale": rng.choice([1.0, 1.0, 0.7, 1.25]),
            "ignored": rng.choice([0.0, 0.0, 0.2, 0.5])}


def _rows(case, what="rows"):
    """Each rank's rows: equal, or falling from the largest to a few (the last of several ranks has none)."""
    n, rows = case["ranks"], case[what]
    if not case["ragged"]:
        return [rows] * n
    return [rows] + [rows * (n - 1 - r) // n for r in range(1, n)]


def _first_rows(case):
    """The index of each rank's first row: replicas hold the same rows, others follow each other."""
    rows = _rows(case)
    return [0 if case["replicas"] else sum(rows[:r]) for r in range(len(rows))]


def _shards(case):
    """The columns of each rank's shard of the vocabulary."""
    return [case["cols"] - (7 * r % 31 if case["uneven"] else 0) for r in range(case["ranks"])]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def _normal(shape, dtype, g, std=1.0, mean=0.0):
    """Normal values made in pieces, so that a 16-bit tensor needs no 32-bit copy of its size."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(std).add_(mean))
    return out


def _row_lists(case, g, std):
    return [_normal((k, case["cols"] + case["pad"]), DTYPES[case["dtype"]], g, std)[:, :case["cols"]]
            for k in _rows(case)]


def _prepare_dropout(case, seed, g, st):
    dt, wt, cols = DTYPES[case["dtype"]], DTYPES[case["wtype"]], case["cols"]
    st["seed"] = (seed * 0x9E3779B97F4A7C15 + 0x1234567) % (1 << 63)
    st["offset"] = 5 + (seed % 1000 << 20)
    # the step's number lives on the device, so that a captured step draws anew when it is replayed
    st["step"] = torch.tensor([seed % 4096], dtype=torch.int64, device="cuda")
    st["first"] = _first_rows(case)
    outs = [torch.empty((k, cols + case["pad"]), dtype=dt, device="cuda")[:, :cols] for k in _rows(case)]
    if case["op"] == "dropout":
        st["xs"] = _row_lists(case, g, 1.0)
        st["residuals"] = _row_lists(case, g, 2.0) if case["residual"] else None
        bias = _normal((cols,), wt, g, 0.3)
        st["biases"] = [bias.clone() for _ in range(case["ranks"])]
        st["ys"] = outs
        return
    st["dys"] = _row_lists(case, g, 0.02)
    st["dxs"] = outs
    st["dbiases"] = [torch.empty(cols, dtype=wt, device="cuda") for _ in range(case["ranks"])]
    if own:
        st["workspace"] = torch.empty(st["B"].arDropoutAddBackwardWorkspace(_rows(case), cols), dtype=torch.uint8,
                                      device="cuda")


def _prepare_logprob(case, g, st):
    """Logits as a model's last product leaves them: a few likely tokens above many unlikely ones, some tokens
    masked out; the targets mostly among the likely ones."""
    dt, rows, shards = DTYPES[case["dtype"]], case["rows"], _shards(case)
    total = sum(shards)
    st["logits"] = [_normal((rows, c), dt, g, 2.5, -1.0) for c in shards]
    st["targets"] = torch.randint(0, total, (rows,), generator=g, device="cuda")
    ignored = torch.rand(rows, generator=g, device="cuda") < case["ignored"]
    st["targets"][ignored] = -100
    first = 0
    for x, c in zip(st["logits"], shards):
        t = st["targets"] - first
        at = ((t >= 0) & (t < c)).nonzero()[:, 0]
        lift = torch.rand(at.numel(), generator=g, device="cuda") * 12.0
        x[at, t[at]] = (x[at, t[at]].float() + lift).to(dt)
        if c > 64:    # a token that may never come
            x[:, c // 2] = torch.where((t == c // 2)[:, None], x[:, c // 2:c // 2 + 1], float("-inf"))[:, 0]
        first += c
    if case["op"] == "logprob":
        st["logp"], st["top"], st["log_sum"] = (torch.empty(rows, device="cuda") for _ in range(3))
        if own:
            st["workspace"] = torch.empty(st["B"].arTokenLogprobWorkspace(rows, shards), dtype=torch.uint8,
                                          device="cuda")
        return
    # the forward pass's statistics, as it keeps them, and the loss's gradient: zero where it was clipped
    top = torch.stack([x.max(1)[0] for x in st["logits"]]).max(0)[0]
    total = torch.zeros(rows, dtype=torch.float64, device="cuda")
    for x in st["logits"]:
        for i in range(0, rows, 2048):
            e = (x[i:i + 2048].float() - top[i:i + 2048, None].float()).mul_(case["scale"]).exp_()
            total[i:i + 2048] += e.sum(1, dtype=torch.float64)
    st["top"], st["log_sum"] = top.float().masked_fill_(ignored, 0.0), total.log().float().masked_fill_(ignored, 0.0)
    dlogp = torch.randn(rows, generator=g, device="cuda")
    st["dlogp"] = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.1, 0.0, dlogp)
    st["dlogits"] = [torch.empty_like(x) for x in st["logits"]]


def _prepare_policy(case, g, st):
    """The tokens' log-probabilities under the policy, the one that sampled them and the reference, after a few
    steps on the same samples; advantages; weights that leave the prompts out."""
    tokens = _rows(case, "tokens")
    for name in ("logps", "olds", "refs", "advantages", "weights", "dlogps"):
        st[name] = []
    for k in tokens:
        old = -torch.rand(k, generator=g, device="cuda").mul_(0.999).add_(1e-3).log_().neg_().mul_(1.5)
        st["olds"].append(old)
        st["logps"].append(old + 0.15 * torch.randn(k, generator=g, device="cuda"))
        st["refs"].append(old + 0.1 * torch.randn(k, generator=g, device="cuda"))
        st["advantages"].append(torch.randn(k, generator=g, device="cuda"))
        st["weights"].append((torch.rand(k, generator=g, device="cuda") < 0.8).float())
        st["dlogps"].append(torch.empty(k, device="cuda"))
    if not case["kl"]:
        st["refs"] = None
    st["stats"] = torch.empty(5, device="cuda")
    if own:
        st["workspace"] = torch.empty(st["B"].arPolicyLossWorkspace(tokens), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case, "stream": torch.cuda.current_stream()}
    if own:
        from ring_allreduce_reduction_amd import binding as B
        st["B"] = B
    if case["op"] in ("dropout", "dropout_backward"):
        _prepare_dropout(case, seed, g, st)
    elif case["op"] in ("logprob", "logprob_backward"):
        _prepare_logprob(case, g, st)
    else:
        _prepare_policy(case, g, st)
    return st


def run(st):
    case = st["case"]
    return {"dropout": _run_dropout, "dropout_backward": _run_dropout_backward, "logprob": _run_logprob,
            "logprob_backward": _run_logprob_backward, "policy": _run_policy}[case["op"]](case, st)


def _high_low(m, v):
    """The upper and lower 32 bits of the product of 32-bit numbers, in parts that stay inside 63 bits."""
    t = m * (v & 0xFFFF)
    u = m * (v >> 16) + (t >> 16)
    return u >> 16, (u & 0xFFFF) << 16 | t & 0xFFFF


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32 of ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
    2011) on 32-bit numbers in int64."""
    for _ in range(10):
        h0, l0 = _high_low(0xD2511F53, c0)
        h1, l1 = _high_low(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c0, c1, c2, c3


def _threshold(case):
    return int(math.floor(case["p"] * 65536 + 0.5))


def _kept(case, st):
    """Which elements of all ranks' rows stay: the number drawn for a row's column c is a 16-bit half of one word
    of the block for its columns 8 (c / 8) to 8 (c / 8) + 7."""
    cols = case["cols"]
    index = torch.cat([torch.arange(f, f + k, device="cuda") for f, k in zip(st["first"], _rows(case))])
    offset = (st["offset"] + st["step"]).view(1, 1)
    groups = torch.arange((cols + 7) // 8, device="cuda")[None, :]
    words = _philox(groups, index[:, None] & 0xFFFFFFFF, offset & 0xFFFFFFFF, offset >> 32,
                    st["seed"] & 0xFFFFFFFF, st["seed"] >> 32)
    words = torch.stack(torch.broadcast_tensors(*words), dim=2)
    halves = torch.stack((words & 0xFFFF, words >> 16), dim=3)
    return halves.reshape(index.numel(), -1)[:, :cols] >= _threshold(case)


def _run_dropout(case, st):
    if own:
        st["B"].arDropoutAdd(st["xs"], st["ys"], case["p"], st["seed"], st["offset"], st["step"], st["biases"],
                             st["residuals"], st["first"], stream=st["stream"])
        return {"y": st["ys"]}
    v = torch.cat(st["xs"]).float() + st["biases"][0].float()
    v = torch.where(_kept(case, st), v * (65536.0 / (65536 - _threshold(case))), 0.0)
    if case["residual"]:
        v = v + torch.cat(st["residuals"]).float()
    return {"y": list(v.to(DTYPES[case["dtype"]]).split(_rows(case)))}


def _run_dropout_backward(case, st):
    if own:
        st["B"].arDropoutAddBackward(st["dys"], st["dxs"], case["p"], st["seed"], st["offset"], st["step"],
                                     st["dbiases"], st["first"], workspace=st["workspace"], stream=st["stream"])
        return {"dx": st["dxs"], "dbias": st["dbiases"]}
    d = torch.cat(st["dys"]).float() * (65536.0 / (65536 - _threshold(case)))
    d = torch.where(_kept(case, st), d, 0.0)
    dbias = d.sum(0).to(DTYPES[case["wtype"]])
    return {"dx": list(d.to(DTYPES[case["dtype"]]).split(_rows(case))), "dbias": [dbias] * case["ranks"]}


def _run_logprob(case, st):
    if own:
        st["B"].arTokenLogprob(st["logits"], st["targets"], st["logp"], st["top"], st["log_sum"], case["scale"],
                               workspace=st["workspace"], stream=st["stream"])
        return {"logp": st["logp"], "top": st["top"], "log_sum": st["log_sum"]}
    x = torch.cat(st["logits"], 1).float()
    top = x.max(1, keepdim=True)[0]
    x = (x - top) * case["scale"]
    log_sum = torch.log(torch.exp(x).sum(1, keepdim=True))
    logp = x.gather(1, st["targets"].clamp(min=0)[:, None]) - log_sum
    out = {"logp": logp, "top": top, "log_sum": log_sum}
    return {k: torch.where(st["targets"] < 0, 0.0, v[:, 0]) for k, v in out.items()}


def _run_logprob_backward(case, st):
    if own:
        st["B"].arTokenLogprobBackward(st["dlogp"], st["logits"], st["targets"], st["top"], st["log_sum"],
                                       st["dlogits"], case["scale"], stream=st["stream"])
        return {"dlogits": st["dlogits"]}
    shards = _shards(case)
    x = torch.cat(st["logits"], 1).float()
    g = torch.where(st["targets"] < 0, 0.0, st["dlogp"] * case["scale"])[:, None]
    p = torch.exp((x - st["top"][:, None]) * case["scale"] - st["log_sum"][:, None])
    d = -p
    at = st["targets"].clamp(min=0)[:, None]
    d = d.scatter(1, at, 1.0 - p.gather(1, at))
    d = torch.where(g == 0.0, 0.0, g * d)
    return {"dlogits": list(d.to(DTYPES[case["dtype"]]).split(shards, 1))}


def _run_policy(case, st):
    if own:
        st["B"].arPolicyLoss(st["logps"], st["olds"], st["advantages"], st["stats"], refs=st["refs"],
                             weights=st["weights"], dlogps=st["dlogps"], clipLow=CLIP_LOW, clipHigh=CLIP_HIGH,
                             klCoef=KL if case["kl"] else 0.0, workspace=st["workspace"], stream=st["stream"])
        return {"stats": st["stats"], "dlogp": st["dlogps"]}
    # 64 bits: ratios next to the clipping bounds, small KL terms, long sums
    logp, old, adv, w = (torch.cat(st[k]).double() for k in ("logps", "olds", "advantages", "weights"))
    ratio = torch.exp(logp - old)
    clipped = ((adv > 0) & (ratio > 1.0 + CLIP_HIGH)) | ((adv < 0) & (ratio < 1.0 - CLIP_LOW))
    loss = -torch.minimum(adv * ratio, adv * ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH))
    grad = torch.where(clipped, 0.0, -adv * ratio)
    kl = torch.zeros_like(loss)
    if case["kl"]:
        d = torch.cat(st["refs"]).double() - logp
        e = torch.exp(d)
        kl = e - d - 1.0
        grad = grad + KL * (1.0 - e)
    total = w.sum()
    part = torch.where(total != 0.0, 1.0 / total, 0.0)
    policy, divergence = (w * loss).sum() * part, (w * kl).sum() * part
    stats = torch.stack((policy + KL * divergence, policy, divergence, (w * clipped).sum() * part, total)).float()
    return {"stats": stats, "dlogp": list((w * part * grad).float().split(_rows(case, "tokens")))}


def work(case):
    if case["op"] in ("dropout", "dropout_backward"):
        e, w, c, n = SIZE[case["dtype"]], SIZE[case["wtype"]], case["cols"], case["ranks"]
        elements = sum(_rows(case)) * c
        if case["op"] == "dropout":
            return {"bytes": (3 if case["residual"] else 2) * elements * e + n * c * w, "flops": 15 * elements}
        return {"bytes": 2 * elements * e + n * c * w, "flops": 14 * elements}
    if case["op"] in ("logprob", "logprob_backward"):
        e, rows = SIZE[case["dtype"]], case["rows"]
        elements = int(rows * (1.0 - case["ignored"])) * sum(_shards(case))
        if case["op"] == "logprob":
            return {"bytes": elements * e + 20 * rows, "flops": 5 * elements}
        return {"bytes": elements * e + rows * sum(_shards(case)) * e + 20 * rows, "flops": 5 * elements}
    tokens = sum(_rows(case, "tokens"))
    return {"bytes": (24 if case["kl"] else 20) * tokens + 20, "flops": 40 * tokens}


def _exact_kept(case, st):
    """The same numbers from products that wrap at 64 bits, a rank at a time."""
    low, offset = 0xFFFFFFFF, st["offset"] + int(st["step"])
    kept = []
    for f, k in zip(st["first"], _rows(case)):
        blocks = (case["cols"] + 7) // 8
        row = torch.arange(f, f + k, device="cuda").repeat_interleave(blocks)
        a, b = torch.arange(blocks, device="cuda").repeat(k), row & low
        c, d = torch.full_like(a, offset & low), torch.full_like(a, offset >> 32)
        for i in range(10):
            p, q = a * 0xD2511F53, c * 0xCD9E8D57
            a = ((q >> 32) & low) ^ b ^ ((st["seed"] + i * 0x9E3779B9) & low)
            c = ((p >> 32) & low) ^ d ^ (((st["seed"] >> 32) + i * 0xBB67AE85) & low)
            b, d = q & low, p & low
        drawn = torch.empty(k, blocks * 8, dtype=torch.int32, device="cuda")
        for j, word in enumerate((a, b, c, d)):
            drawn[:, 2 * j::8] = (word % 65536).view(k, blocks).int()
            drawn[:, 2 * j + 1::8] = word.div(65536, rounding_mode="floor").view(k, blocks).int()
        kept.append(drawn[:, :case["cols"]] >= _threshold(case))
    return kept


def exact(case, seed):
    """From the definitions in 64 bits: dropout as a product with the mask, log-probabilities as a difference to
    the logarithm of the summed exponentials, the policy loss by its cases."""
    st = prepare(case, seed)
    if case["op"] in ("dropout", "dropout_backward"):
        rate = 1.0 - _threshold(case) / 65536.0
        masks = [k.double().div_(rate) for k in _exact_kept(case, st)]
        if case["op"] == "dropout":
            ys = [m.mul_(x.double().add_(b.double())) for m, x, b in zip(masks, st["xs"], st["biases"])]
            if st["residuals"] is not None:
                ys = [y.add_(r.double()) for y, r in zip(ys, st["residuals"])]
            return {"y": ys}
        dxs = [m.mul_(dy.double()) for m, dy in zip(masks, st["dys"])]
        dbias = sum(torch.ones(d.shape[0], dtype=torch.float64, device="cuda") @ d for d in dxs)
        return {"dx": dxs, "dbias": [dbias for _ in dxs]}
    if case["op"] == "logprob":
        out = {"logp": [], "top": [], "log_sum": []}
        for i in range(0, case["rows"], 1024):
            t = st["targets"][i:i + 1024]
            z = torch.cat([x[i:i + 1024].double() for x in st["logits"]], 1).mul_(case["scale"])
            whole = torch.logsumexp(z, 1)
            top = z.amax(1)
            logp = z[torch.arange(t.numel(), device="cuda"), t.clamp(min=0)] - whole
            for name, v in (("logp", logp), ("top", top / case["scale"]), ("log_sum", whole - top)):
                out[name].append(v.masked_fill(t < 0, 0.0))
        return {k: torch.cat(v) for k, v in out.items()}
    if case["op"] == "logprob_backward":
        parts, first = [], 0
        scale = case["scale"]
        live = (st["targets"] >= 0).double()
        g = (st["dlogp"].double() * scale * live).unsqueeze(1)
        shift = (st["log_sum"].double() + scale * st["top"].double()).unsqueeze(1)
        for x in st["logits"]:
            d = x.double().mul_(scale).sub_(shift).exp_().mul_(-g).mul_(live.unsqueeze(1))
            t = st["targets"] - first
            at = ((t >= 0) & (t < x.shape[1])).nonzero()[:, 0]
            d[at, t[at]] += g[at, 0]
            d.masked_fill_(g == 0.0, 0.0)
            parts.append(d)
            first += x.shape[1]
        return {"dlogits": parts}
    logp, old, adv, w = (torch.cat(st[k]).double() for k in ("logps", "olds", "advantages", "weights"))
    change = logp - old
    up = (adv > 0) & (change > math.log1p(CLIP_HIGH))
    down = (adv < 0) & (change < math.log1p(-CLIP_LOW))
    bound = torch.where(up, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW)
    free = ~(up | down)
    loss = -adv * torch.where(free, change.exp(), bound)
    grad = -adv * change.exp() * free
    kl = torch.zeros_like(loss)
    if case["kl"]:
        d = torch.cat(st["refs"]).double() - logp
        kl = torch.expm1(d) - d
        grad = grad - KL * torch.expm1(d)
    total = float(w.sum())
    over = 1.0 / total if total else 0.0
    policy, divergence = float(torch.dot(w, loss)) * over, float(torch.dot(w, kl)) * over
    stats = torch.tensor([policy + KL * divergence, policy, divergence, float((w * ~free).sum()) * over, total],
                         dtype=torch.float64, device="cuda")
    return {"stats": stats, "dlogp": list((w * grad * over).split(_rows(case, "tokens")))}
