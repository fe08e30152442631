"""A fine-tuning step as its operators are used together: two data-parallel groups, each with its layer's product and
the vocabulary cut over three ranks.  AllReduce of the partial products, dropout with bias and residual, layer norm,
logits, log-probabilities, policy loss over both groups' tokens; and back, to the clipped gradients of every weight.
Against torch's autograd in 64 bits on the CPU."""
import op_util as ou
import pytest
import step_util as su
import torch

pytestmark = pytest.mark.gpu

GROUPS, RANKS, INNER, HIDDEN, SHARDS = 2, 3, 20, 48, [50, 61, 39]
TOKENS = [37, 22]
P, SEED, OFFSET, EPS = 0.25, 77, 3 << 20, 1e-5
LOW, HIGH, KL, SCALE = 0.2, 0.28, 0.1, 1.25


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from ring_allreduce_reduction_amd import binding
    binding.lib()
    return binding


def data():
    g = torch.Generator().manual_seed(5)
    d = {"a": [[torch.randn(t, INNER, generator=g) for _ in range(RANKS)] for t in TOKENS],
         "w1": [torch.randn(INNER, HIDDEN, generator=g) * 0.2 for _ in range(RANKS)],
         "bias": torch.randn(HIDDEN, generator=g) * 0.3, "gamma": 1 + 0.2 * torch.randn(HIDDEN, generator=g),
         "beta": 0.1 * torch.randn(HIDDEN, generator=g), "w2": [torch.randn(HIDDEN, c, generator=g) * 0.3 for c in SHARDS],
         "res": [torch.randn(t, HIDDEN, generator=g) for t in TOKENS],
         "targets": [torch.randint(0, sum(SHARDS), (t,), generator=g) for t in TOKENS],
         "adv": [torch.randn(t, generator=g) for t in TOKENS], "noise": [0.2 * torch.randn(t, generator=g) for t in TOKENS],
         "noise2": [0.2 * torch.randn(t, generator=g) for t in TOKENS]}
    for t in d["targets"]:
        t[:5] = -100                                   # the prompt
    d["weight"] = [(t >= 0).float() for t in d["targets"]]
    return d


def in_64_bits(d):
    leaf = {k: d[k].double().requires_grad_() for k in ("bias", "gamma", "beta")}
    w1 = [w.double().requires_grad_() for w in d["w1"]]
    w2 = [w.double().requires_grad_() for w in d["w2"]]
    total, old, ref, first = 0.0, [], [], 0
    for g in range(GROUPS):
        x = sum(a.double() @ w for a, w in zip(d["a"][g], w1))
        kept = su.drawn(TOKENS[g], first, HIDDEN, SEED, OFFSET) >= su.threshold(P)
        first += TOKENS[g]
        y = d["res"][g].double() + torch.where(kept, (x + leaf["bias"]) * su.scale_of(P), 0.0)
        h = torch.nn.functional.layer_norm(y, (HIDDEN,), leaf["gamma"], leaf["beta"], EPS)
        logits = torch.cat([h @ w for w in w2], 1) * SCALE
        t = d["targets"][g]
        logp = torch.log_softmax(logits, 1).gather(1, t.clamp(min=0)[:, None])[:, 0]
        old.append((logp.detach() + d["noise"][g]).float())
        ref.append((logp.detach() + d["noise2"][g]).float())
        ratio = torch.exp(logp - old[g].double())
        assert ((ratio - (1 + HIGH)).abs() > 1e-4).all() and ((ratio - (1 - LOW)).abs() > 1e-4).all()
        adv = d["adv"][g].double()
        loss = -torch.minimum(adv * ratio, adv * ratio.clamp(1 - LOW, 1 + HIGH))
        diff = ref[g].double() - logp
        total = total + (d["weight"][g].double() * (loss + KL * (torch.exp(diff) - diff - 1))).sum()
    loss = total / sum(w.double().sum() for w in d["weight"])
    loss.backward()
    return loss.item(), [leaf["bias"].grad, leaf["gamma"].grad, leaf["beta"].grad] + [w.grad for w in w1 + w2], old, ref


def test_a_step_forward_and_back(B):
    d = data()
    loss, want, old, ref = in_64_bits(d)
    cuda = lambda ts: [t.cuda() for t in ts]   # noqa: E731
    w1, w2 = cuda(d["w1"]), cuda(d["w2"])
    bias, gamma, beta = ([d[k].cuda() for _ in TOKENS] for k in ("bias", "gamma", "beta"))
    new = lambda ts: [torch.full_like(t, float("nan")) for t in ts]   # noqa: E731
    acts = [cuda(a) for a in d["a"]]
    res, targets = cuda(d["res"]), cuda(d["targets"])
    torch.cuda.synchronize()
    with B.Comm(RANKS, 4, "simple") as comm:
        xs = []
        for g in range(GROUPS):
            parts = [a @ w for a, w in zip(acts[g], w1)]
            outs = new(parts)
            comm.allreduce(parts, outs)
            xs.append(outs[0])
        ys, hs = new(xs), new(xs)
        means, rstds = ([torch.empty(t, device="cuda") for t in TOKENS] for _ in range(2))
        B.arDropoutAdd(xs, ys, P, SEED, OFFSET, None, bias, res)
        B.arLayerNorm(ys, hs, gamma, beta, means, rstds, eps=EPS)
        logits = [[h @ w for w in w2] for h in hs]
        logp, top, lsum = ([torch.full((t,), float("nan"), device="cuda") for t in TOKENS] for _ in range(3))
        for g in range(GROUPS):
            B.arTokenLogprob(logits[g], targets[g], logp[g], top[g], lsum[g], SCALE)
        stats, dlogp = torch.empty(5, device="cuda"), new(logp)
        B.arPolicyLoss(logp, cuda(old), cuda(d["adv"]), stats, cuda(ref), cuda(d["weight"]), dlogp, LOW, HIGH, KL)
        dhs, dw2 = [], [torch.zeros_like(w) for w in w2]
        for g in range(GROUPS):
            B.arTokenLogprobBackward(dlogp[g], logits[g], targets[g], top[g], lsum[g], logits[g], SCALE)   # in place
            parts = [x @ w.t() for x, w in zip(logits[g], w2)]
            outs = new(parts)
            comm.allreduce(parts, outs)
            dhs.append(outs[0])
            for k in range(RANKS):
                dw2[k] += hs[g].t() @ logits[g][k]
        dys, dgamma, dbeta = new(ys), new(gamma), new(beta)
        B.arLayerNormBackward(dhs, ys, means, rstds, gamma, dys, dgamma, dbeta)
        dxs, dbias = new(xs), new(bias)
        B.arDropoutAddBackward(dys, dxs, P, SEED, OFFSET, None, dbias)
        dw1 = [sum(acts[g][k].t() @ dxs[g] for g in range(GROUPS)) for k in range(RANKS)]
    torch.cuda.synchronize()
    got = [dbias[0], dgamma[0], dbeta[0]] + dw1 + dw2
    assert torch.equal(dbias[0], dbias[1]) and torch.equal(dgamma[0], dgamma[1])
    # ten steps, each off by at most the 200 terms of its longest sum times U of what it adds up
    size = max(w.abs().max().item() for w in want)
    assert abs(stats[0].item() - loss) <= 2000 * ou.U * (1 + abs(loss))
    for a, b in zip(got, want):
        assert (a.double().cpu() - b).abs().max().item() <= 2000 * ou.U * size
    # the gradients' norm, and clipping in place
    norm = torch.empty(1, device="cuda")
    whole = torch.cat([w.reshape(-1) for w in want]).norm().item()
    with B.TensorList(got, got) as lst:
        B.arGradClip(lst, norm, whole / 2, eps=0.0)
        torch.cuda.synchronize()
    assert abs(norm.item() - whole) <= 2000 * ou.U * size * sum(w.numel() for w in want) ** 0.5
    for a, b in zip(got, want):
        assert (a.double().cpu() - b / 2).abs().max().item() <= 4000 * ou.U * size
