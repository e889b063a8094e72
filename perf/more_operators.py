"""Cases of the operators at the two ends of a training step: losses from sharded logits (token
log-probabilities, a clipped policy loss with a KL term, a preference loss of pairs), forward and
with their gradient, and the AdamW step over many tensors with states in 32 or in 8 bits.

``run`` computes a case in elementary torch operations in 32 bits, or (``own``) by the calls that a
program makes of this framework.  ``exact`` computes it in 64 bits, apart from ``run``'s plain form.
"""
import functools
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
# logits: `tokens` rows over a vocabulary that `ranks` ranks share, `cols` columns each (what a
#   column-parallel projection leaves); logits / grad: their types; temperature: logits are divided
#   by it; masked: share of tokens without a target; entropy: the rows' entropies too
def _logits(kind, tokens, cols, ranks=1, logits="bf16", grad="bf16", temperature=1.0, masked=0.0, entropy=False):
    return {"kind": kind, "tokens": tokens, "cols": cols, "ranks": ranks, "logits": logits, "grad": grad,
            "temperature": temperature, "masked": masked, "entropy": entropy}


# policy loss: kl: weight of the KL term against reference log-probabilities (0: none); bonus: weight
#   of the entropy; weighted: tokens have weights
def _policy(tokens, cols, ranks=1, kl=0.0, bonus=0.0, weighted=False, **more):
    return {**_logits("policy", tokens, cols, ranks, **more), "kl": kl, "bonus": bonus, "weighted": weighted}


# preference loss: `pairs` pairs of packed sequences of ragged lengths (`lengths` seeds them)
def _preference(tokens, cols, pairs, ranks=1, loss="sigmoid", beta=0.1, smoothing=0.0, average=False, lengths=0,
                **more):
    return {**_logits("preference", tokens, cols, ranks, **more), "pairs": pairs, "loss": loss, "beta": beta,
            "smoothing": smoothing, "average": average, "lengths": lengths}


# AdamW: shapes: "layer" (an MLP layer's projections on `ranks` ranks: hidden x ffn, gate and up in
#   one) or "ragged" (`count` tensors of odd sizes, `total` elements or so, `lengths` seeds them);
#   param / grad: types; master: bf16 parameters have fp32 masters; bits: of the states; clip: the
#   gradients' norm is taken first and clipped to this (0: neither); stochastic: bf16 parameters
#   without masters are rounded stochastically
def _adamw(shapes, total=0, count=0, hidden=0, ffn=0, ranks=1, param="bf16", grad="bf16", master=True, bits=32,
           clip=0.0, stochastic=False, lengths=0, step=100):
    return {"kind": "adamw", "shapes": shapes, "total": total, "count": count, "hidden": hidden, "ffn": ffn,
            "ranks": ranks, "param": param, "grad": grad, "master": master, "bits": bits, "clip": clip,
            "stochastic": stochastic, "lengths": lengths, "step": step}


def listed():
    return [
        # scoring the last tokens of a short answer: latency
        {"name": "logprob_16", **_logits("logprob", 16, 32000)},
        # a reference model's log-probabilities over 4096 tokens, the vocabulary on 8 ranks
        {"name": "logprob_4k", **_logits("logprob", 4096, 16384, 8, entropy=True)},
        # supervised training on 32-bit logits over an odd vocabulary, a tenth of it prompt
        {"name": "nll_train_1000", **_logits("nll_train", 1000, 50001, logits="f32", masked=0.1)},
        # a policy update on one short answer: latency
        {"name": "policy_48", **_policy(48, 16000, 2, kl=0.05)},
        # a policy update over 4096 tokens, the vocabulary on 8 ranks, KL against the reference
        {"name": "policy_4k", **_policy(4096, 16384, 8, kl=0.04, masked=0.25)},
        # odd sizes, temperature, entropy bonus and token weights, everything in 32 bits
        {"name": "policy_2047", **_policy(2047, 10671, 3, bonus=0.01, weighted=True, logits="f32", grad="f32",
                                          temperature=0.7, masked=0.3)},
        # two pairs of short answers
        {"name": "preference_333", **_preference(333, 32000, 2, lengths=3, masked=0.4)},
        # eight pairs, the vocabulary on 4 ranks, smoothed labels
        {"name": "preference_8k", **_preference(8192, 8192, 8, 4, smoothing=0.1, lengths=4, masked=0.3)},
        # norm weights of a model: many tiny tensors, latency
        {"name": "adamw_64_vectors", **_adamw("ragged", total=200000, count=64, param="f32", grad="f32", master=False,
                                              lengths=1)},
        # an 8B-shaped MLP layer on 4 ranks, 32-bit masters and states, gradients clipped
        {"name": "adamw_layer", **_adamw("layer", hidden=4096, ffn=14336, ranks=4, clip=1.0)},
        # the same with states in 8 bits
        {"name": "adamw8_layer", **_adamw("layer", hidden=4096, ffn=14336, ranks=4, bits=8, clip=1.0)},
        # ragged tensors in bf16 alone, stochastically rounded, 8-bit states, 32-bit gradients
        {"name": "adamw8_ragged", **_adamw("ragged", total=3000000, count=37, grad="f32", master=False, bits=8,
                                           stochastic=True, lengths=2)},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["logprob", "nll_train", "policy", "policy", "preference", "adamw", "adamw"])
    if kind == "adamw":
        bits, param = rng.choice([32, 8]), rng.choice(["bf16", "bf16", "f32"])
        master = param == "bf16" and rng.random() < 0.6
        how = {"bits": bits, "param": param, "master": master, "grad": rng.choice(["bf16", "f32"]),
               "clip": rng.choice([0.0, 1.0]), "stochastic": param == "bf16" and not master and rng.random() < 0.7,
               "lengths": rng.randrange(1 << 20), "step": _log_int(rng, 1, 100000)}
        if rng.random() < 0.3:
            return _adamw("layer", hidden=256 * rng.randint(2, 16), ffn=512 * rng.randint(2, 28),
                          ranks=rng.choice([1, 2, 4]), **how)
        return _adamw("ragged", total=_log_int(rng, 1, 1 << 26), count=_log_int(rng, 1, 500), **how)
    ranks = rng.choice([1, 1, 2, 3, 4, 8])
    cols = rng.choice([64 * rng.randint(2, 512), _log_int(rng, 2, 65536)])
    tokens = _log_int(rng, 1, 16384)
    while ranks * tokens * cols > 1 << 28:
        tokens = max(1, tokens * 2 // 3)
        cols = cols * 5 // 6
    how = {"logits": rng.choice(["bf16", "bf16", "f32"]), "grad": rng.choice(["bf16", "bf16", "f32"]),
           "temperature": rng.choice([1.0, 1.0, round(rng.uniform(0.5, 2.0), 2)]),
           "masked": rng.choice([0.0, 0.25, round(rng.random(), 2)])}
    if kind == "policy":
        return _policy(tokens, cols, ranks, kl=rng.choice([0.0, 0.05]), bonus=rng.choice([0.0, 0.01]),
                       weighted=rng.random() < 0.5, **how)
    if kind == "preference":
        return _preference(tokens, cols, rng.randint(1, 16), ranks, loss=rng.choice(["sigmoid", "squared", "hinge"]),
                           beta=rng.choice([0.05, 0.1, 0.5]), smoothing=rng.choice([0.0, 0.1]),
                           average=rng.random() < 0.4, lengths=rng.randrange(1 << 20), **how)
    return _logits(kind, tokens, cols, ranks, entropy=kind == "logprob" and rng.random() < 0.5, **how)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
BLOCK = 256   # elements that share the ranges of 8-bit states


def _sizes(case):
    if case["shapes"] == "layer":
        f = case["ffn"] // case["ranks"]
        return [n for _ in range(case["ranks"]) for n in (2 * f * case["hidden"], case["hidden"] * f)]
    rng = random.Random(case["lengths"])
    w = [math.exp(rng.uniform(0, 4)) for _ in range(case["count"])]
    return [max(1, int(case["total"] * x / sum(w))) for x in w]


def _offsets(case):
    rng = random.Random(case["lengths"])
    t, n = case["tokens"], 2 * case["pairs"]
    return [0] + sorted(rng.randint(0, t) for _ in range(n - 1)) + [t]


def _pitched(ranks, rows, cols, dtype, device):
    """[ranks, rows, cols] whose rows start on 16-byte boundaries (the framework's row pitch)."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((ranks, rows, -(-cols // per) * per), dtype=dtype, device=device)[..., :cols]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(1000003 * (seed + 1) + 29)
    s = {"case": case}
    (_prepare_adamw if case["kind"] == "adamw" else _prepare_logits)(s, g, dev)
    if own:
        s["ctx"] = _context(dev.index)
        if case["kind"] == "adamw":
            import overlapped_tensor_gemm_gb300 as fo
            s["group"] = fo.AdamWTensors(*(_tensors(s, x) for x in ("w", "g", "m", "v")),
                                         master=_tensors(s, "master") if case["master"] else None,
                                         m_scale=_tensors(s, "m_scale"), v_range=_tensors(s, "v_range"))
            s["m_list"], s["v_list"] = _tensors(s, "m_out"), _tensors(s, "v_out")
    return s


def _prepare_logits(s, g, dev):
    case = s["case"]
    p, t, c = case["ranks"], case["tokens"], case["cols"]
    rand = lambda *shape: torch.rand(shape, generator=g, device=dev)  # noqa: E731
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    s["targets"] = (rand(t) * (p * c)).long().clamp_(max=p * c - 1)
    s["logits"] = _pitched(p, t, c, DTYPES[case["logits"]], dev)
    for r in range(p):
        z = randn(t, c) * 2.0
        # the model has learnt something: a token's own logit stands out by a random amount
        here = (s["targets"] >= r * c) & (s["targets"] < (r + 1) * c)
        z[here, s["targets"][here] - r * c] += 2.0 + 5.0 * rand(int(here.sum()))
        s["logits"][r].copy_(z)
        del z
    s["dlogits"] = _pitched(p, t, c, DTYPES[case["grad"]], dev)
    one = lambda n=t: torch.empty(n, dtype=torch.float32, device=dev)  # noqa: E731
    s["logp"], s["lse"], s["entropy"] = one(), one(), one() if case["entropy"] else None
    if case["kind"] in ("policy", "preference"):
        # what the policy that sampled, and a reference, gave these tokens: near the present policy's
        scaled = [s["logits"][r].float() / case["temperature"] for r in range(p)]
        lse = torch.logsumexp(torch.stack([torch.logsumexp(z, -1) for z in scaled]), 0)
        own_logit = torch.zeros(t, device=dev)
        for r, z in enumerate(scaled):
            here = ((s["targets"] >= r * c) & (s["targets"] < (r + 1) * c)).nonzero()[:, 0]
            own_logit[here] = z[here, s["targets"][here] - r * c]
        del scaled
        logp = own_logit - lse
        s["old"] = logp + 0.15 * randn(t)
        s["ref"] = logp + 0.3 * randn(t)
    if case["kind"] == "policy":
        s["advantages"] = randn(t)
        s["weights"] = 0.25 + rand(t) if case["weighted"] else None
        s["stats"] = one(4)
    if case["kind"] == "preference":
        s["offsets"] = torch.tensor(_offsets(case), dtype=torch.int32, device=dev)
        s["loss"], s["margins"] = one(1), one(case["pairs"])
    s["targets"] = torch.where(rand(t) < case["masked"], -1, s["targets"]).to(torch.int32)
    s["dlogp"] = torch.where(s["targets"] < 0, 0.0, -1.0 / max(1, t)) if case["kind"] == "nll_train" else None


def _prepare_adamw(s, g, dev):
    """One buffer for each kind of value; a tensor starts on a block's boundary."""
    case = s["case"]
    s["sizes"] = _sizes(case)
    s["blocks"] = [-(-n // BLOCK) for n in s["sizes"]]
    nb = sum(s["blocks"])
    n = nb * BLOCK
    randn = lambda k: torch.randn(k, generator=g, device=dev)  # noqa: E731
    count = torch.tensor(s["blocks"], device=dev)
    first = torch.cumsum(count, 0) - count
    s["of"] = torch.repeat_interleave(torch.arange(len(s["blocks"]), device=dev), count)   # a block's tensor
    s["at"] = torch.arange(nb, device=dev) - first[s["of"]]                                # its place in it
    live = (s["at"][:, None] * BLOCK + torch.arange(BLOCK, device=dev) <
            torch.tensor(s["sizes"], device=dev)[s["of"]][:, None]).reshape(-1)
    # rows of a weight differ in scale, and so do their gradients
    wide = torch.exp2(randn(nb)).repeat_interleave(BLOCK) * live
    master = randn(n) * 0.02 * live
    s["w"] = master.to(DTYPES[case["param"]])
    s["master"] = master if case["master"] else None
    s["g"] = (randn(n) * 1e-3 * wide).to(DTYPES[case["grad"]])
    m, v = randn(n) * 3e-4 * wide, (1e-3 * wide).square() * torch.exp2(randn(n))
    s["m_scale"] = s["v_range"] = s["m_out"] = s["v_out"] = None
    if case["bits"] == 8:
        s["m_scale"] = (m.reshape(-1, BLOCK).abs().amax(1) / 448).clamp(min=1e-30)
        s["m"] = (m.reshape(-1, BLOCK) / s["m_scale"][:, None]).to(torch.float8_e4m3fn).reshape(-1)
        low = torch.where(v > 0, v.log2(), math.inf).reshape(-1, BLOCK).amin(1)
        top = torch.where(v > 0, v.log2(), -math.inf).reshape(-1, BLOCK).amax(1)
        gap = ((top - low) / 254).clamp(min=1e-6)
        s["v_range"] = torch.stack([low, gap], 1).reshape(-1)
        code = 1 + ((v.log2().reshape(-1, BLOCK) - low[:, None]) / gap[:, None]).round()
        s["v"] = torch.where(v.reshape(-1, BLOCK) > 0, code, torch.zeros_like(code)).to(torch.uint8).reshape(-1)
        s["m_out"], s["v_out"] = (torch.zeros(n, dtype=torch.bfloat16, device=dev) for _ in range(2))
    else:
        s["m"], s["v"] = m, v
    s["norm"] = torch.zeros(1, device=dev)
    s["seed"] = int(torch.randint(0, 1 << 62, (1,), generator=g, device=dev))


PER_BLOCK = {"m_scale": 1, "v_range": 2}


def _tensors(s, name):
    """The tensors of one kind, as views of their buffer."""
    if s[name] is None:
        return None
    per, out, at = PER_BLOCK.get(name), [], 0
    for n, b in zip(s["sizes"], s["blocks"]):
        out.append(s[name][at * (per or BLOCK):][:b * per if per else n])
        at += b
    return out


@functools.lru_cache(maxsize=None)
def _context(device):
    """The program's one context on a device."""
    import overlapped_tensor_gemm_gb300 as fo
    return fo.Context(device)


HYPER = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}
CLIP_LOW, CLIP_HIGH = 0.2, 0.28


# ---------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------
def _run_own(s):
    case, ctx = s["case"], s["ctx"]
    if case["kind"] == "adamw":
        if case["clip"]:
            ctx.grad_norm(s["group"], s["norm"])
        ctx.adamw_step(s["group"], step=case["step"], norm=s["norm"] if case["clip"] else None, max_norm=case["clip"],
                       stochastic=case["stochastic"], seed=s["seed"], **HYPER)
        if case["bits"] == 8:
            ctx.adamw_unpack(s["group"], s["m_list"], s["v_list"])
        return _adamw_outputs(s)
    logits, dlogits = list(s["logits"].unbind(0)), list(s["dlogits"].unbind(0))
    scale = 1.0 / case["temperature"]
    if case["kind"] == "logprob":
        ctx.token_logprobs(logits, s["targets"], s["logp"], lse=s["lse"], entropy=s["entropy"], scale=scale)
        return {x: s[x] for x in ("logp", "lse", "entropy") if s[x] is not None}
    if case["kind"] == "nll_train":
        ctx.token_logprobs(logits, s["targets"], s["logp"], lse=s["lse"], scale=scale)
        ctx.token_logprobs_backward(logits, s["targets"], s["lse"], s["dlogp"], dlogits, scale=scale)
        return {x: s[x] for x in ("logp", "lse", "dlogits")}
    if case["kind"] == "policy":
        ctx.policy_loss(logits, s["targets"], s["advantages"], s["stats"], old_logp=s["old"],
                        ref_logp=s["ref"] if case["kl"] else None, weights=s["weights"], logp=s["logp"],
                        dlogits=dlogits, clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=case["kl"],
                        entropy_coef=case["bonus"], scale=scale)
        return {x: s[x] for x in ("stats", "logp", "dlogits")}
    ctx.preference_loss(logits, s["targets"], s["offsets"], s["loss"], ref_logp=s["ref"], logp=s["logp"],
                        margins=s["margins"], dlogits=dlogits, kind=case["loss"], beta=case["beta"],
                        label_smoothing=case["smoothing"], average=case["average"], scale=scale)
    return {x: s[x] for x in ("loss", "margins", "logp", "dlogits")}


def _adamw_outputs(s):
    names = ("w", "master") + (("m_out", "v_out") if s["case"]["bits"] == 8 else ("m", "v"))
    return {x: s[x] for x in names + (("norm",) if s["case"]["clip"] else ()) if s[x] is not None}


# ---------------------------------------------------------------------------------------------
# the plain forms: 32 bits, rounded once at the end
# ---------------------------------------------------------------------------------------------
def _rows(s):
    """(z - max z, log sum exp of it, the target's column of it, which tokens count, max z) in 32 bits."""
    case = s["case"]
    z = torch.cat(list(s["logits"].unbind(0)), 1).float()
    if case["temperature"] != 1.0:
        z = z.mul_(1.0 / case["temperature"])
    top = z.amax(1, keepdim=True)
    z = z.sub_(top)
    total = z.exp().sum(1)
    counted = s["targets"] >= 0
    at = s["targets"].clamp(min=0).long()
    return z, total.log(), z.gather(1, at[:, None])[:, 0], counted, top[:, 0]


def _entropy(z, log_total):
    return log_total - (z.exp() * z).sum(1) / log_total.exp()


def _gradient(s, z, log_total, counted, dlogp, dentropy=None):
    """dlogits [ranks, tokens, cols]: d logp = 1[target] - p; d entropy = -p (log p + entropy)."""
    case = s["case"]
    zero = torch.zeros_like(log_total)
    dlogp = torch.where(counted, dlogp, zero)
    add = -dlogp[:, None]
    if dentropy is not None:
        entropy = _entropy(z, log_total)
        add = add - torch.where(counted, dentropy, zero)[:, None] * (z - log_total[:, None] + entropy[:, None])
    d = z.sub_(log_total[:, None]).exp_().mul_(add)
    d.scatter_add_(1, s["targets"].clamp(min=0).long()[:, None], dlogp[:, None])
    if case["temperature"] != 1.0:
        d = d.mul_(1.0 / case["temperature"])
    p, c = case["ranks"], case["cols"]
    return d.reshape(-1, p, c).permute(1, 0, 2).to(DTYPES[case["grad"]])


def _pair_loss(case, gap):
    """Loss of each pair by its gap, and its derivative."""
    beta, x = case["beta"], case["beta"] * gap
    if case["loss"] == "sigmoid":
        return (-x).clamp(min=0) + (-x.abs()).exp().log1p(), -beta / (1 + x.exp())
    if case["loss"] == "squared":
        return (gap - 0.5 / beta).square(), 2 * (gap - 0.5 / beta)
    return (1 - x).clamp(min=0), torch.where(x < 1, -beta, 0.0)


def _plain_logits(s):
    case = s["case"]
    z, log_total, own_z, counted, top = _rows(s)
    zero = torch.zeros_like(log_total)
    logp = torch.where(counted, own_z - log_total, zero)
    out = {"logp": logp}
    if case["kind"] in ("logprob", "nll_train"):
        out["lse"] = torch.where(counted, top + log_total, zero)
        if case["entropy"]:
            out["entropy"] = torch.where(counted, _entropy(z, log_total), zero)
        if case["kind"] == "nll_train":
            out["dlogits"] = _gradient(s, z, log_total, counted, s["dlogp"])
        return out
    if case["kind"] == "policy":
        weight = torch.ones_like(logp) if s["weights"] is None else s["weights"]
        weight = torch.where(counted, weight, zero)
        weight = weight / weight.sum().clamp(min=1e-30)
        ratio = (logp - s["old"]).exp()
        a = s["advantages"]
        free, held = ratio * a, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * a
        clipped = held < free
        loss, dlogp = -torch.minimum(free, held), torch.where(clipped, zero, -free)
        kl = zero
        if case["kl"]:
            x = s["ref"] - logp
            kl = x.expm1() - x
            loss, dlogp = loss + case["kl"] * kl, dlogp - case["kl"] * x.expm1()
        entropy = _entropy(z, log_total)
        loss = loss - case["bonus"] * entropy
        out["stats"] = torch.stack([(weight * x).sum() for x in (loss, kl, clipped.float(), entropy)])
        out["dlogits"] = _gradient(s, z, log_total, counted, weight * dlogp,
                                   -case["bonus"] * weight if case["bonus"] else None)
        return out
    pairs, off = case["pairs"], s["offsets"].long()
    seq = torch.bucketize(torch.arange(case["tokens"], device=logp.device), off[1:], right=True).clamp(max=2 * pairs - 1)
    ratio = torch.where(counted, logp - s["ref"], zero).double()
    score = torch.zeros(2 * pairs, dtype=torch.float64, device=logp.device).index_add_(0, seq, ratio)
    share = torch.ones_like(score)
    if case["average"]:
        share = 1 / torch.zeros_like(score).index_add_(0, seq, counted.double()).clamp(min=1)
        score = score * share
    gap = (score[:pairs] - score[pairs:]).float()
    x, eps = case["beta"] * gap, case["smoothing"]
    loss, dgap = _pair_loss(case, gap)
    if eps:  # some labels are the wrong way round
        loss2, dgap2 = _pair_loss(case, -gap)
        loss, dgap = (1 - eps) * loss + eps * loss2, (1 - eps) * dgap - eps * dgap2
    out["loss"], out["margins"] = loss.double().mean().float()[None], x
    coef = torch.cat([dgap, -dgap]) / pairs * share.float()
    out["dlogits"] = _gradient(s, z, log_total, counted, coef[seq])
    return out


def _mix(x):
    """32 bits scattered (whole numbers in 64-bit tensors)."""
    x = (x ^ (x >> 16)) * 0x7FEB352D & 0xFFFFFFFF
    x = (x ^ (x >> 15)) * 0x846CA68B & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_words(s):
    """[blocks, BLOCK] 32-bit numbers from the seed, the step, a tensor's place in the list, a block's in
    the tensor and an element's in the block."""
    dev, seed = s["of"].device, s["seed"]
    word = lambda v: torch.tensor(v & 0xFFFFFFFF, dtype=torch.int64, device=dev)  # noqa: E731
    key = _mix(_mix(word(seed) ^ _mix(word(s["case"]["step"]))) ^ word(seed >> 32))
    block = _mix((_mix((key + s["of"]) & 0xFFFFFFFF) + s["at"]) & 0xFFFFFFFF)
    return _mix((block[:, None] + torch.arange(BLOCK, device=dev) * 0x9E3779B9) & 0xFFFFFFFF)


def _unpacked(s):
    m = s["m"].float().reshape(-1, BLOCK) * s["m_scale"][:, None]
    low, gap = s["v_range"].reshape(-1, 2, 1).unbind(1)
    code = s["v"].float().reshape(-1, BLOCK)
    return m.reshape(-1), torch.where(code > 0, torch.exp2(low + (code - 1) * gap), torch.zeros_like(code)).reshape(-1)


def _pack(s, m, v, words):
    """8 bits, rounded up or down at random so that the mean is the value: m as e4m3 times a scale for each
    block, v as 0 or one of 255 values between the block's smallest and largest, evenly spaced in log2."""
    m, v = m.reshape(-1, BLOCK), v.reshape(-1, BLOCK)
    scale = m.abs().amax(1, keepdim=True) / 448
    x = torch.where(scale > 0, m / scale, torch.zeros_like(m))
    size = x.abs().clamp(max=448)
    lift = torch.where(size < 2.0 ** -6, 2.0 ** -6, 0.0)  # below it e4m3's steps stay 2^-9 wide
    bits = (size + lift).view(torch.int32) + ((words & 0xFFFF) << 4).to(torch.int32) & -0x100000
    s["m"].copy_(torch.copysign(bits.view(torch.float32) - lift, x).to(torch.float8_e4m3fn).reshape(-1))
    s["m_scale"].copy_(scale[:, 0])
    some = v > 0
    lg = v.log2()
    top = torch.where(some, lg, -math.inf).amax(1, keepdim=True)
    low = torch.maximum(torch.where(some, lg, math.inf).amin(1, keepdim=True), top - 24)
    none = ~some.any(1, keepdim=True)
    low, gap = (torch.where(none, 0.0, x) for x in (low, (top - low) / 254))
    y = torch.where(gap > 0, (lg - low) / gap, torch.zeros_like(lg)).clamp(0, 254)
    whole = y.floor()
    part = y - whole
    part = part - 0.5 * math.log(2) * gap * part * (1 - part)  # the mean of the values, not of their logarithms
    up = (words >> 16).float() * 2.0 ** -16 < part
    s["v"].copy_(torch.where(some, 1 + whole + up, 0.0).to(torch.uint8).reshape(-1))
    s["v_range"].copy_(torch.cat([low, gap], 1).reshape(-1))


def _plain_adamw(s):
    case, h = s["case"], HYPER
    g = s["g"].float()
    if case["clip"]:
        s["norm"].copy_(g.double().square().sum().sqrt())
        g = g * (case["clip"] / s["norm"]).clamp(max=1.0)
    eight = case["bits"] == 8
    m, v = _unpacked(s) if eight else (s["m"], s["v"])
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g.square()
    w = (s["master"] if case["master"] else s["w"]).float()
    fix1, fix2 = 1 - h["beta1"] ** case["step"], 1 - h["beta2"] ** case["step"]
    w = w - h["lr"] * (h["weight_decay"] * w + (m / fix1) / ((v / fix2).sqrt() + h["eps"]))
    words = _random_words(s) if eight or case["stochastic"] else None
    if case["master"]:
        s["master"].copy_(w)
    if case["stochastic"]:
        low = (words * 0x9E3779B9 & 0xFFFFFFFF) >> 16
        w = (w.view(torch.int32) + low.reshape(-1).to(torch.int32) & -0x10000).view(torch.float32)
    s["w"].copy_(w)
    if eight:
        _pack(s, m, v, words)
        for name, x in zip(("m_out", "v_out"), _unpacked(s)):
            s[name].copy_(x)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_outputs(s)


def run(s):
    if own:
        return _run_own(s)
    return _plain_adamw(s) if s["case"]["kind"] == "adamw" else _plain_logits(s)


# ---------------------------------------------------------------------------------------------
# 64 bits, from the definitions: gradients by differentiating the forward definition
# ---------------------------------------------------------------------------------------------
def _exact_rows(s, lo, hi, grad):
    """Leaf, log-probabilities of the targets, log-sum-exp and entropy of rows lo..hi."""
    case = s["case"]
    leaf = torch.cat([s["logits"][r, lo:hi] for r in range(case["ranks"])], 1).double().requires_grad_(grad)
    z = leaf / case["temperature"]
    lse = torch.logsumexp(z, 1)
    lp = z - lse[:, None]
    logp = lp[torch.arange(hi - lo, device=lp.device), s["targets"][lo:hi].clamp(min=0).long()]
    return leaf, logp, lse, -(lp.exp() * lp).sum(1)


def _exact_logits(s):
    case = s["case"]
    t, v = case["tokens"], case["ranks"] * case["cols"]
    slab = max(1, (1 << 27) // v)
    parts = [(lo, min(t, lo + slab)) for lo in range(0, t, slab)]
    with torch.no_grad():
        logp, lse, entropy = (torch.cat(x) for x in zip(*(_exact_rows(s, lo, hi, False)[1:] for lo, hi in parts)))
    counted = s["targets"] >= 0
    only = lambda x: torch.where(counted, x, torch.zeros_like(x))  # noqa: E731
    logp = only(logp)
    out = {"logp": logp}
    if case["kind"] == "logprob":
        return {**out, "lse": only(lse), **({"entropy": only(entropy)} if case["entropy"] else {})}
    # the loss as a function of the tokens' log-probabilities and entropies
    lp, h = logp.clone().requires_grad_(), only(entropy).requires_grad_()
    if case["kind"] == "nll_train":
        out["lse"] = only(lse)
        loss = (s["dlogp"].double() * lp).sum() + 0 * h.sum()
    elif case["kind"] == "policy":
        w = only(torch.ones_like(logp) if s["weights"] is None else s["weights"].double())
        w = w / w.sum() if bool(w.sum() > 0) else w
        rho, a = torch.exp(lp - s["old"].double()), s["advantages"].double()
        near = torch.where(a >= 0, torch.clamp(rho, max=1 + CLIP_HIGH), torch.clamp(rho, min=1 - CLIP_LOW))
        per = -near * a
        kl = torch.zeros_like(lp)
        if case["kl"]:
            d = s["ref"].double() - lp
            kl = torch.exp(d) - d - 1
        loss = (w * (per + case["kl"] * kl - case["bonus"] * h)).sum()
        out["stats"] = torch.stack([loss, (w * kl).sum(), (w * (near != rho)).sum(), (w * h).sum()]).detach()
    else:
        n, b = case["pairs"], _offsets(case)
        score = []
        for lo, hi in zip(b[:-1], b[1:]):
            d = ((lp[lo:hi] - s["ref"][lo:hi].double()) * counted[lo:hi]).sum()
            score.append(d / max(1, int(counted[lo:hi].sum())) if case["average"] else d)
        gap = torch.stack(score[:n]) - torch.stack(score[n:])
        x, eps = case["beta"] * gap, case["smoothing"]
        each = {"sigmoid": lambda d: -torch.nn.functional.logsigmoid(case["beta"] * d),
                "squared": lambda d: (d - 1 / (2 * case["beta"])) ** 2,
                "hinge": lambda d: torch.relu(1 - case["beta"] * d)}[case["loss"]]
        each = (1 - eps) * each(gap) + eps * each(-gap)
        loss = each.mean() + 0 * h.sum()
        out["loss"], out["margins"] = loss.detach()[None], x.detach()
    dlp, dh = torch.autograd.grad(loss, [lp, h], allow_unused=True)
    dlp, dh = only(dlp), only(torch.zeros_like(lp) if dh is None else dh)
    out["dlogits"] = torch.empty((case["ranks"], t, case["cols"]), dtype=torch.float64, device=logp.device)
    for lo, hi in parts:
        leaf, a, _, b = _exact_rows(s, lo, hi, True)
        seed = (a * dlp[lo:hi]).sum() + ((b * dh[lo:hi]).sum() if bool(dh.any()) else 0)
        d, = torch.autograd.grad(seed, leaf)
        out["dlogits"][:, lo:hi] = d.reshape(hi - lo, case["ranks"], case["cols"]).transpose(0, 1)
    return out


def _scatter32(x):
    for shift, factor in ((16, 0x7FEB352D), (15, 0x846CA68B)):
        x = ((x ^ (x >> shift)) * factor) % (1 << 32)
    return x ^ (x >> 16)


def _exact_adamw(s):
    case, h = s["case"], HYPER
    g = s["g"].double()
    out = {}
    if case["clip"]:
        norm = torch.linalg.vector_norm(g)
        out["norm"] = norm[None]
        g = g * min(1.0, case["clip"] / float(norm))
    rows = lambda x: x.reshape(-1, BLOCK)  # noqa: E731
    if case["bits"] == 8:
        m = (rows(s["m"].double()) * s["m_scale"].double()[:, None]).reshape(-1)
        lo, gap = s["v_range"].double().reshape(-1, 2).T[:, :, None]
        code = rows(s["v"].double())
        v = ((code > 0) * 2.0 ** (lo + gap * (code - 1))).reshape(-1)
    else:
        m, v = s["m"].double(), s["v"].double()
    m, v = torch.lerp(g, m, h["beta1"]), torch.lerp(g * g, v, h["beta2"])
    w = (s["master"] if case["master"] else s["w"]).double()
    t = case["step"]
    w = w * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * (m / (1 - h["beta1"] ** t)) / (
        torch.sqrt(v / (1 - h["beta2"] ** t)) + h["eps"])
    if case["master"]:
        out["master"] = w
    if case["bits"] == 32:
        return {**out, "w": w, "m": m, "v": v}
    dev = w.device
    seed_low, seed_high = s["seed"] % (1 << 32), s["seed"] >> 32
    key = _scatter32(_scatter32(seed_low ^ _scatter32(t % (1 << 32))) ^ seed_high)
    one = _scatter32((_scatter32((key + s["of"]) % (1 << 32)) + s["at"]) % (1 << 32))
    r = _scatter32((one[:, None] + 0x9E3779B9 * torch.arange(BLOCK, device=dev)) % (1 << 32))
    # e4m3: steps of 2^(e-3) between 2^e and 2^(e+1), of 2^-9 below 2^-6
    m, v = rows(m), rows(v)
    scale = m.abs().amax(1, keepdim=True) / 448
    x = torch.where(scale > 0, m.abs() / scale, torch.zeros_like(m))
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    q = torch.floor(x / step + (r % 65536) / 65536.0) * step
    out["m_out"] = (torch.sign(m) * q * scale).reshape(-1)
    lg = torch.log2(torch.where(v > 0, v, torch.ones_like(v)))
    top = torch.where(v > 0, lg, torch.full_like(lg, -1e9)).amax(1, keepdim=True)
    low = torch.where(v > 0, lg, torch.full_like(lg, 1e9)).amin(1, keepdim=True).clamp(min=top - 24)
    gap = (top - low) / 254
    y = torch.where(gap > 0, (lg - low) / gap, torch.zeros_like(lg)).clamp(0, 254)
    f = y - torch.floor(y)
    f = f * (1 - math.log(2) / 2 * gap * (1 - f))
    y = torch.floor(y) + ((r >> 16) / 65536.0 < f)
    out["v_out"] = torch.where(v > 0, torch.exp2(low + gap * y), torch.zeros_like(v)).reshape(-1)
    return {**out, "w": w}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_adamw(s) if case["kind"] == "adamw" else _exact_logits(s)


def work(case):
    if case["kind"] == "adamw":
        n, blocks = sum(_sizes(case)), sum(-(-x // BLOCK) for x in _sizes(case))
        size = {x: 2 if case[x] == "bf16" else 4 for x in ("param", "grad")}
        # a clipped gradient is read for its norm and again for the step
        each = size["grad"] * (2 if case["clip"] else 1) + size["param"] + (8 if case["master"] else size["param"])
        each += 16 if case["bits"] == 32 else 4 + 4   # the states as values (16 bits each) are outputs too
        return {"bytes": n * each + (24 * blocks if case["bits"] == 8 else 0), "flops": 20 * n}
    n, t = case["tokens"] * case["cols"] * case["ranks"], case["tokens"]
    read = n * (2 if case["logits"] == "bf16" else 4)
    wrote = n * (2 if case["grad"] == "bf16" else 4)
    if case["kind"] == "logprob":
        return {"bytes": read + 4 * t * (4 if case["entropy"] else 3), "flops": 4 * n}
    # masked rows are not read, but their gradients are written
    return {"bytes": int(read * (1 - case["masked"])) + wrote + 4 * t * 6, "flops": 10 * n}
