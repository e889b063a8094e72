"""Cases of the training operators around the projections: attention with row statistics and its
backward pass, norms before and after a block with gate and residual, rotary positions.

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
# attention: P independent ranks (each its own heads over all tokens, as in the attention block),
#   tokens queries, prefix further keys before them, docs packed sequences (1: one sequence)
def _attn(kind, tokens, heads, kv_heads, dim=128, ranks=1, causal=True, prefix=0, docs=1, lengths=0):
    return {"kind": kind, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "ranks": ranks,
            "causal": causal, "prefix": prefix, "docs": docs, "lengths": lengths}


# norms: ranks token slices of `rows` rows; res / act / par: types of the residual stream, of the
#   block's output and the normed activations, and of the weights; gate: none, row (one learned
#   vector) or token (a gate for every token); post: the block's output is normed; pre: the next
#   block's input is
def _norm(kind, rows, hidden, ranks=1, res="bf16", act="bf16", par="bf16", gate="row", post=True, pre=True,
          alpha=1.0):
    return {"kind": kind, "rows": rows, "hidden": hidden, "ranks": ranks, "res": res, "act": act, "par": par,
            "gate": gate, "post": post, "pre": pre, "alpha": alpha}


# rotary positions: `rows` tokens of `heads` heads; the first rot of dim dimensions turn; scaling: none,
#   linear, banded (low frequencies slowed, high kept) or ramped (with an amplitude); start: the first
#   token's position; scattered: positions given one by one
def _rope(kind, rows, heads, dim=128, rot=128, layout="half", dtype="bf16", scaling="none", start=0,
          scattered=False, base=10000.0):
    return {"kind": kind, "rows": rows, "heads": heads, "dim": dim, "rot": rot, "layout": layout, "dtype": dtype,
            "scaling": scaling, "start": start, "scattered": scattered, "base": base}


def listed():
    return [
        # a rank's heads of one short prompt: latency
        {"name": "attn_fwd_128", **_attn("attn_fwd", 128, 8, 8)},
        # evaluation of an 8K sequence, 32 query heads on 8 key/value heads
        {"name": "attn_fwd_8k", **_attn("attn_fwd", 8192, 32, 8)},
        # a training step on one short sequence of odd length
        {"name": "attn_train_333", **_attn("attn_train", 333, 4, 4)},
        # the attention block's configuration: 4 ranks of 8 heads over 4096 tokens
        {"name": "attn_train_4x4k", **_attn("attn_train", 4096, 8, 8, ranks=4)},
        # packed documents of ragged lengths, heads of 64 dimensions
        {"name": "attn_train_packed", **_attn("attn_train", 8000, 16, 4, dim=64, docs=23, lengths=5)},
        # the longest sequence of the sweep, one rank's share of 32 heads
        {"name": "attn_train_16k", **_attn("attn_train", 16384, 8, 2)},
        # the norms around one block for a handful of tokens: latency
        {"name": "norm_fwd_16", **_norm("norm_fwd", 16, 4096, gate="none", post=False)},
        # 8 ranks' slices of 16K tokens at width 8192, 32-bit residual stream
        {"name": "norm_fwd_8x2k", **_norm("norm_fwd", 2048, 8192, ranks=8, res="f32", alpha=0.5)},
        # backward of the same with the residual stream in 16 bits
        {"name": "norm_bwd_8x2k", **_norm("norm_bwd", 2048, 8192, ranks=8)},
        # backward at a width that is no multiple of a vector, gates for every token, 32-bit weights
        {"name": "norm_bwd_1000", **_norm("norm_bwd", 1000, 1001, gate="token", par="f32", alpha=1.25)},
        # the query and key heads of 16K tokens far into a long context
        {"name": "rope_fwd_16k", **_rope("rope_fwd", 16384, 40, scaling="banded", base=500000.0, start=114688)},
        # gradients of interleaved pairs in part of the head, positions given, 32 bits
        {"name": "rope_bwd_1023", **_rope("rope_bwd", 1023, 9, dim=96, rot=64, layout="interleaved", dtype="f32",
                                          scaling="ramped", start=1 << 20, scattered=True)},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attn_fwd", "attn_train", "attn_train", "norm_fwd", "norm_bwd", "rope_fwd", "rope_bwd"])
    if kind.startswith("attn"):
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 4, 5])
        ranks = rng.choice([1, 1, 2, 4])
        tokens = _log_int(rng, 1, 16384)
        docs = rng.choice([1, 1, 1, rng.randint(2, 40)])
        prefix = _log_int(rng, 1, 4096) if docs == 1 and rng.random() < 0.25 else 0
        most = 8 * 16384 * 16384  # scores of the largest listed case
        while ranks * heads * tokens * (tokens + prefix) > most:
            tokens = tokens * 2 // 3
        return _attn(kind, tokens, heads, kv, dim=rng.choice([64, 128, 128]), ranks=ranks,
                     causal=rng.random() < 0.75, prefix=prefix, docs=docs, lengths=rng.randrange(1 << 20))
    if kind.startswith("norm"):
        hidden = rng.choice([64 * rng.randint(2, 128), _log_int(rng, 16, 16384)])
        rows = _log_int(rng, 1, 16384)
        ranks = rng.choice([1, 1, 2, 4, 8])
        while rows * ranks * hidden > 16384 * 8192:
            rows = rows * 2 // 3
        pre = rng.random() < 0.9
        return _norm(kind, rows, hidden, ranks=ranks, res=rng.choice(["bf16", "f32"]),
                     act=rng.choice(["bf16", "bf16", "f32"]), par=rng.choice(["bf16", "f32"]),
                     gate=rng.choice(["none", "row", "token"]), post=rng.random() < 0.7 or not pre, pre=pre,
                     alpha=rng.choice([1.0, 1.0, round(rng.uniform(0.25, 2.0), 3)]))
    dim = rng.choice([64, 128, 128, 2 * rng.randint(8, 128)])
    rot = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
    heads = _log_int(rng, 1, 64)
    rows = _log_int(rng, 1, 32768)
    while rows * heads * dim > 16384 * 40 * 128:
        rows = rows * 2 // 3
    return _rope(kind, rows, heads, dim=dim, rot=rot, layout=rng.choice(["half", "interleaved"]),
                 dtype=rng.choice(["bf16", "bf16", "f32"]), scaling=rng.choice(["none", "linear", "banded", "ramped"]),
                 start=rng.choice([0, rng.randrange(1 << 21)]), scattered=rng.random() < 0.4,
                 base=rng.choice([10000.0, 500000.0, 1000000.0]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _offsets(case):
    """Boundaries of the packed sequences: random cuts, an empty sequence among them now and then."""
    rng = random.Random(case["lengths"])
    n, t = case["docs"], case["tokens"]
    return [0] + sorted(rng.randint(0, t) for _ in range(n - 1)) + [t]


def _pairs(case):
    """(query, key) pairs of one head that the mask keeps."""
    if case["docs"] > 1:
        b = _offsets(case)
        lens = [(b[i + 1] - b[i], b[i + 1] - b[i]) for i in range(case["docs"])]
    else:
        lens = [(case["tokens"], case["tokens"] + case["prefix"])]
    return sum(lq * (lk - lq) + lq * (lq + 1) // 2 if case["causal"] else lq * lk for lq, lk in lens)


def _padded(ranks, rows, cols, dtype, device):
    """[ranks, rows, cols] whose rows start on 16-byte boundaries (the framework's row pitch)."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((ranks, rows, -(-cols // per) * per), dtype=dtype, device=device)[..., :cols]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(1000003 * (seed + 1) + 17)

    def randn(ranks, rows, cols, dtype, std=1.0, mean=0.0):
        t = _padded(ranks, rows, cols, dtype, dev)
        t.copy_(torch.randn((ranks, rows, cols), generator=g, device=dev) * std + mean)
        return t

    s = {"case": case}
    if case["kind"].startswith("attn"):
        p, t, h, kv, d = case["ranks"], case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        tk = t + case["prefix"]
        # the projection's output holds queries, keys and values side by side; keys of a longer
        # context come from a buffer of their own
        bf = torch.bfloat16
        if tk == t:
            qkv = randn(p, t, (h + 2 * kv) * d, bf)
            grad = torch.empty_like(qkv)
            cut = [h * d, kv * d, kv * d]
            s["q"], s["k"], s["v"] = torch.split(qkv, cut, dim=2)
            s["dq"], s["dk"], s["dv"] = torch.split(grad, cut, dim=2)
        else:
            s["q"], s["k"], s["v"] = randn(p, t, h * d, bf), randn(p, tk, kv * d, bf), randn(p, tk, kv * d, bf)
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in "qkv")
        s["do"] = randn(p, t, h * d, bf)
        s["o"] = torch.empty((p, t, h * d), dtype=bf, device=dev)
        s["lse"] = _padded(p, h, t, torch.float32, dev)
        s["offsets"] = torch.tensor(_offsets(case), dtype=torch.int32, device=dev) if case["docs"] > 1 else None
    elif case["kind"].startswith("norm"):
        p, m, c = case["ranks"], case["rows"], case["hidden"]
        res, act, par = DTYPES[case["res"]], DTYPES[case["act"]], DTYPES[case["par"]]
        s["r"] = randn(p, m, c, res, 2.0)       # the residual stream (backward: after the block)
        s["y"] = randn(p, m, c, act, 0.7)       # the block's output
        s["w_post"] = randn(1, 1, c, par, 0.1, 1.0)[0, 0] if case["post"] else None
        s["w_pre"] = randn(1, 1, c, par, 0.1, 1.0)[0, 0] if case["pre"] else None
        s["gate"] = {"none": lambda: None, "row": lambda: randn(1, 1, c, par, 0.3, 0.5)[0, 0],
                     "token": lambda: randn(p, m, c, par, 0.3, 0.5)}[case["gate"]]()
        s["r_out"] = _padded(p, m, c, res, dev)
        s["x"] = _padded(p, m, c, act, dev) if case["pre"] else None
        if case["kind"] == "norm_bwd":
            s["dx"] = randn(p, m, c, act) if case["pre"] else None
            s["dr_out"] = randn(p, m, c, res)
            s["dr"], s["dy"] = _padded(p, m, c, res, dev), _padded(p, m, c, act, dev)
            one = lambda: torch.empty(c, dtype=torch.float32, device=dev)  # noqa: E731
            s["dw_post"] = one() if case["post"] else None
            s["dw_pre"] = one() if case["pre"] else None
            s["dgate"] = {"none": lambda: None, "row": one, "token": lambda: _padded(p, m, c, par, dev)}[case["gate"]]()
    else:
        m, h, d = case["rows"], case["heads"], case["dim"]
        s["x"] = randn(1, m, h * d, DTYPES[case["dtype"]])
        s["y"] = _padded(1, m, h * d, DTYPES[case["dtype"]], dev)
        s["positions"] = None
        if case["scattered"]:
            s["positions"] = (case["start"] + torch.randint(0, 65536, (m,), generator=g, device=dev)).to(torch.int32)
    if own:
        s["ctx"] = _context(dev.index)
        if case["kind"].startswith("rope"):
            import overlapped_tensor_gemm_gb300 as fo
            s["table"] = fo.RopeTable(case["rot"], base=case["base"], **SCALINGS[case["scaling"]])
    return s


@functools.lru_cache(maxsize=None)
def _context(device):
    """The program's one context on a device."""
    import overlapped_tensor_gemm_gb300 as fo
    return fo.Context(device)


# ---------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------
def _ranks(t):
    return None if t is None else list(t.unbind(0))


def _run_own(s):
    case, ctx = s["case"], s["ctx"]
    if case["kind"].startswith("attn"):
        q, k, v, o, lse = (_ranks(s[x]) for x in ("q", "k", "v", "o", "lse"))
        how = {"heads": case["heads"], "kv_heads": case["kv_heads"], "head_dim": case["dim"],
               "causal": case["causal"], "q_offsets": s["offsets"]}
        ctx.attn_forward(q, k, v, o, lse, **how)
        if case["kind"] == "attn_fwd":
            return {"o": s["o"], "lse": s["lse"]}
        ctx.attn_backward(q, k, v, o, lse, _ranks(s["do"]), _ranks(s["dq"]), _ranks(s["dk"]), _ranks(s["dv"]), **how)
        return {x: s[x] for x in ("o", "lse", "dq", "dk", "dv")}
    if case["kind"].startswith("norm"):
        token = case["gate"] == "token"
        how = {"w_post": s["w_post"], "gate": _ranks(s["gate"]) if token else s["gate"], "w_pre": s["w_pre"],
               "residual_scale": case["alpha"], "eps": EPS}
        if case["kind"] == "norm_fwd":
            ctx.norm_residual(_ranks(s["r"]), _ranks(s["y"]), _ranks(s["r_out"]), _ranks(s["x"]), **how)
            return {"r_out": s["r_out"], **({"x": s["x"]} if case["pre"] else {})}
        ctx.norm_residual_backward(_ranks(s["r"]), _ranks(s["y"]), _ranks(s["dx"]), _ranks(s["dr_out"]),
                                   _ranks(s["dr"]), _ranks(s["dy"]), dw_post=s["dw_post"],
                                   dgate=_ranks(s["dgate"]) if token else s["dgate"], dw_pre=s["dw_pre"], **how)
        return {x: s[x] for x in ("dr", "dy", "dw_post", "dgate", "dw_pre") if s[x] is not None}
    call = ctx.rope if case["kind"] == "rope_fwd" else ctx.rope_backward
    call(_ranks(s["x"]), _ranks(s["y"]), s["table"], head_dim=case["dim"], layout=case["layout"],
         positions=None if s["positions"] is None else [s["positions"]], start=case["start"])
    return {"y": s["y"]}


# ---------------------------------------------------------------------------------------------
# the plain forms: 32 bits, rounded once at the end
# ---------------------------------------------------------------------------------------------
EPS = 1e-6
SCALINGS = {
    "none": {},
    "linear": {"scaling": "linear", "factor": 4.0},
    "banded": {"scaling": "banded", "factor": 8.0, "low_factor": 1.0, "high_factor": 4.0, "original_length": 8192},
    "ramped": {"scaling": "ramped", "factor": 16.0, "beta_fast": 32.0, "beta_slow": 1.0, "original_length": 4096},
}


def _mask(case, offsets, device):
    """[queries, keys] truth values: the pairs that attend."""
    t, tk = case["tokens"], case["tokens"] + case["prefix"]
    i = torch.arange(t, device=device)[:, None]
    j = torch.arange(tk, device=device)[None, :]
    keep = j <= i + case["prefix"] if case["causal"] else torch.ones((t, tk), dtype=torch.bool, device=device)
    if offsets is not None:
        doc = torch.bucketize(torch.arange(t, device=device), offsets[1:].long(), right=True)
        keep = keep & (doc[:, None] == doc[None, :])
    return keep


def _heads(t, heads, groups, dim):
    """[ranks, tokens, heads * dim] -> [ranks, groups, heads per group, tokens, dim] in 32 bits."""
    p, n = t.shape[:2]
    return t.float().reshape(p, n, groups, heads // groups, dim).permute(0, 2, 3, 1, 4)


def _back(t, like):
    p, a, b, n, d = t.shape
    return t.permute(0, 3, 1, 2, 4).reshape(p, n, a * b * d).to(like.dtype)


def _plain_attn(s):
    case = s["case"]
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    q, k, v = _heads(s["q"], h, kv, d), _heads(s["k"], kv, kv, d), _heads(s["v"], kv, kv, d)
    scale = 1.0 / math.sqrt(d)
    keep = _mask(case, s["offsets"], q.device)
    sc = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~keep, -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1).flatten(1, 2)
    p = p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    out = {"o": _back(p @ v, s["q"]), "lse": lse}
    if case["kind"] == "attn_train":
        do = _heads(s["do"], h, kv, d)
        dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
        ds = do @ v.transpose(-1, -2)
        delta = (ds * p).sum(-1, keepdim=True)
        ds = ds.sub_(delta).mul_(p).mul_(scale)
        out["dq"] = _back(ds @ k, s["q"])
        out["dk"] = _back((ds.transpose(-1, -2) @ q).sum(2, keepdim=True), s["k"])
        out["dv"] = _back(dv, s["v"])
    return out


def _plain_norm(s):
    case = s["case"]
    y = s["y"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    if s["w_post"] is not None:
        inv_y = (y.square().mean(-1, keepdim=True) + EPS).rsqrt()
        u = y * inv_y
        z = u * s["w_post"].float()
    else:
        z = y
    if case["kind"] == "norm_fwd":
        r = case["alpha"] * s["r"].float() + gate * z
        out = {"r_out": r.to(s["r"].dtype)}
        if case["pre"]:
            x = r * (r.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["w_pre"].float()
            out["x"] = x.to(s["y"].dtype)
        return out
    out = {}
    r, dr = s["r"].float(), s["dr_out"].float()
    if case["pre"]:
        inv = (r.square().mean(-1, keepdim=True) + EPS).rsqrt()
        n, dx = r * inv, s["dx"].float()
        out["dw_pre"] = (dx * n).flatten(0, 1).sum(0)
        dn = dx * s["w_pre"].float()
        dr = dr + inv * (dn - n * (dn * n).mean(-1, keepdim=True))
    out["dr"] = (case["alpha"] * dr).to(s["r"].dtype)
    if case["gate"] == "row":
        out["dgate"] = (dr * z).flatten(0, 1).sum(0)
    elif case["gate"] == "token":
        out["dgate"] = (dr * z).to(s["gate"].dtype)
    dz = dr * gate
    if s["w_post"] is not None:
        out["dw_post"] = (dz * u).flatten(0, 1).sum(0)
        du = dz * s["w_post"].float()
        dz = inv_y * (du - u * (du * u).mean(-1, keepdim=True))
    out["dy"] = dz.to(s["y"].dtype)
    return out


def _frequencies(case, device):
    """(radians per position of each pair, amplitude) in 64 bits."""
    rot, how = case["rot"], SCALINGS[case["scaling"]]
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    f = case["base"] ** (-2.0 * i / rot)
    kind = how.get("scaling")
    if kind == "linear":
        f = f / how["factor"]
    elif kind == "banded":  # wavelengths above length/low: slowed; below length/high: kept; between: mixed
        turns = how["original_length"] * f / (2 * math.pi)
        mix = ((turns - how["low_factor"]) / (how["high_factor"] - how["low_factor"])).clamp(0, 1)
        f = (1 - mix) * f / how["factor"] + mix * f
    elif kind == "ramped":  # by pair index: kept up to the pair that turns beta_fast times, slowed from beta_slow on
        pair = lambda b: rot * math.log(how["original_length"] / (2 * math.pi * b)) / (2 * math.log(case["base"]))  # noqa: E731
        low, high = max(math.floor(pair(how["beta_fast"])), 0), min(math.ceil(pair(how["beta_slow"])), rot - 1)
        mix = 1 - ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = (1 - mix) * f / how["factor"] + mix * f
        return f, 0.1 * math.log(how["factor"]) + 1.0
    return f, 1.0


def _positions(s):
    case = s["case"]
    if s["positions"] is not None:
        return s["positions"].double()
    return case["start"] + torch.arange(case["rows"], dtype=torch.float64, device=s["x"].device)


def _plain_rope(s):
    case = s["case"]
    m, h, d, rot = case["rows"], case["heads"], case["dim"], case["rot"]
    f, amp = _frequencies(case, s["x"].device)
    angle = _positions(s)[:, None] * f[None, :]  # 64 bits: far positions
    cos, sin = (amp * angle.cos()).float()[:, None, :], (amp * angle.sin()).float()[:, None, :]
    if case["kind"] == "rope_bwd":
        sin = -sin
    x = s["x"].float().reshape(m, h, d)
    turn, rest = x[..., :rot], x[..., rot:]
    if case["layout"] == "half":
        a, b = turn[..., :rot // 2], turn[..., rot // 2:]
        turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return {"y": torch.cat([turn, rest], -1).reshape(1, m, h * d).to(s["x"].dtype)}


def run(s):
    if own:
        return _run_own(s)
    kind = s["case"]["kind"]
    return _plain_attn(s) if kind.startswith("attn") else _plain_norm(s) if kind.startswith("norm") else _plain_rope(s)


# ---------------------------------------------------------------------------------------------
# 64 bits, from the definitions: gradients by differentiating the forward definition
# ---------------------------------------------------------------------------------------------
def _exact_attn(s):
    case = s["case"]
    h, kv, d, t = case["heads"], case["kv_heads"], case["dim"], case["tokens"]
    bounds = _offsets(case) if case["docs"] > 1 else [0, t]
    train = case["kind"] == "attn_train"
    out = {x: torch.zeros(s[x].shape, dtype=torch.float64, device=s[x].device)
           for x in (("o", "lse", "dq", "dk", "dv") if train else ("o", "lse"))}
    for p in range(case["ranks"]):
        for lo, hi in zip(bounds[:-1], bounds[1:]):
            klo, khi = lo, hi + case["prefix"]
            if lo == hi:
                continue
            for head in range(h):
                cq, ck = slice(head * d, head * d + d), slice(head // (h // kv) * d, (head // (h // kv) + 1) * d)
                leaf = [s[x][p, a:b, c].double().requires_grad_(train)
                        for x, a, b, c in (("q", lo, hi, cq), ("k", klo, khi, ck), ("v", klo, khi, ck))]
                w = leaf[0] @ leaf[1].T / math.sqrt(d)
                if case["causal"]:
                    w = w + torch.full_like(w, -math.inf).triu(1 + case["prefix"])
                o = torch.softmax(w, -1) @ leaf[2]
                out["o"][p, lo:hi, cq] = o.detach()
                out["lse"][p, head, lo:hi] = torch.logsumexp(w.detach(), -1)
                if train:
                    dq, dk, dv = torch.autograd.grad(o, leaf, s["do"][p, lo:hi, cq].double())
                    out["dq"][p, lo:hi, cq] = dq
                    out["dk"][p, klo:khi, ck] += dk
                    out["dv"][p, klo:khi, ck] += dv
    return out


def _exact_norm(s):
    case = s["case"]
    rms = lambda t: (t * t).mean(-1, keepdim=True).add(EPS).sqrt()  # noqa: E731
    need = case["kind"] == "norm_bwd"
    leaf = {x: s[x].double().requires_grad_(need) for x in ("r", "y", "w_post", "w_pre", "gate") if s[x] is not None}

    def branch():
        z = leaf["y"] if "w_post" not in leaf else leaf["y"] / rms(leaf["y"]) * leaf["w_post"]
        return z * leaf["gate"] if "gate" in leaf else z

    if not need:
        r = case["alpha"] * leaf["r"] + branch()
        return {"r_out": r, **({"x": r / rms(r) * leaf["w_pre"]} if case["pre"] else {})}
    out, dr = {}, s["dr_out"].double()
    if case["pre"]:
        x = leaf["r"] / rms(leaf["r"]) * leaf["w_pre"]
        add, out["dw_pre"] = torch.autograd.grad(x, [leaf["r"], leaf["w_pre"]], s["dx"].double())
        dr = dr + add
    out["dr"] = case["alpha"] * dr
    names = [x for x in ("y", "w_post", "gate") if x in leaf]
    for x, g in zip(names, torch.autograd.grad(branch(), [leaf[x] for x in names], dr)):
        out["d" + x] = g
    return out


def _exact_rope(s):
    case = s["case"]
    m, h, d, rot = case["rows"], case["heads"], case["dim"], case["rot"]
    how, freq, amp = SCALINGS[case["scaling"]], [], 1.0
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(case["base"]))
        slow = f / how.get("factor", 1.0)
        if how.get("scaling") == "linear":
            f = slow
        elif how.get("scaling") == "banded":
            wave = 2 * math.pi / f
            lo, hi, n = how["low_factor"], how["high_factor"], how["original_length"]
            if wave > n / lo:
                f = slow
            elif wave >= n / hi:
                mix = (n / wave - lo) / (hi - lo)
                f = (1 - mix) * slow + mix * f
        elif how.get("scaling") == "ramped":
            amp = 1.0 + math.log(how["factor"]) / 10
            at = [rot * math.log(how["original_length"] / (how[b] * 2 * math.pi)) / (2 * math.log(case["base"]))
                  for b in ("beta_fast", "beta_slow")]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
            part = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = part * slow + (1 - part) * f
        freq.append(f)
    sign = -1.0 if case["kind"] == "rope_bwd" else 1.0
    angle = sign * _positions(s)[:, None] * torch.tensor(freq, dtype=torch.float64, device=s["x"].device)
    turn = torch.polar(torch.full_like(angle, amp), angle)[:, None, :]
    x = s["x"].double().reshape(m, h, d)
    y = x.clone()
    first, second = ((slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half"
                     else (slice(0, rot, 2), slice(1, rot, 2)))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return {"y": y.reshape(1, m, h * d)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("attn"):
        # over about 20 seconds in 64 bits
        if case["ranks"] * case["heads"] * case["tokens"] * (case["tokens"] + case["prefix"]) > 3 * 10 ** 9:
            return None
        return _exact_attn(s)
    return _exact_norm(s) if case["kind"].startswith("norm") else _exact_rope(s)


def work(case):
    if case["kind"].startswith("attn"):
        p, t, h, kv, d = case["ranks"], case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        q, k = 2 * p * t * h * d, 2 * p * (t + case["prefix"]) * kv * d
        fwd = {"bytes": 2 * q + 2 * k + 4 * p * h * t, "flops": 4 * d * _pairs(case) * h * p}
        if case["kind"] == "attn_fwd":
            return fwd
        # gradients: dO read, dQ, dK and dV written; five products, the scores again among them
        return {"bytes": fwd["bytes"] + 2 * q + 2 * k, "flops": 14 * d * _pairs(case) * h * p}
    if case["kind"].startswith("norm"):
        n = case["ranks"] * case["rows"] * case["hidden"]
        size = {x: 2 if case[x] == "bf16" else 4 for x in ("res", "act", "par")}
        gate = size["par"] * n if case["gate"] == "token" else 0
        vectors = (case["post"] + case["pre"] + (case["gate"] == "row")) * case["hidden"]
        if case["kind"] == "norm_fwd":
            return {"bytes": n * (2 * size["res"] + size["act"] * (1 + case["pre"])) + gate + size["par"] * vectors,
                    "flops": 10 * n}
        return {"bytes": n * (3 * size["res"] - (0 if case["pre"] else size["res"]) + size["act"] * (2 + case["pre"]))
                + 2 * gate + (4 + size["par"]) * vectors, "flops": 30 * n}
    n = case["rows"] * case["heads"] * case["dim"]
    return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + (4 * case["rows"] if case["scattered"] else 0),
            "flops": 3 * n}
